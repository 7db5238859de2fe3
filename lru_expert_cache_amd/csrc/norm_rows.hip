// Root-mean-square norm: rows that a workgroup's registers hold, read once.
//
// Bound by HBM: 8192 rows of 7168, bf16, called over and over: with a 32-bit
// stream forward 126 us (5.6 TB/s read and written), backward 182 (5.2, the
// join of the weight's gradient included); with a bf16 stream forward, codes and
// y, 107 us (4.9).  A copy of 2 GiB moves 4.9 TB/s.  Persistent workgroups
// take the rows of the backward pass in turn, so that 512 parts of the
// weight's gradient are left to add up; the forward pass has a workgroup for
// each row.  Pieces of four columns beside 32-bit rows (lanes then lie side by
// side in either) were 1 to 3% faster forward and no faster backward: not kept.
//
// A thread has PIECES pieces of eight neighbouring columns.  The piece that
// would pass the row's end is taken from its last eight columns instead: what
// it shares with the piece before is left out of the sums, and written twice
// with the same value.
#include "norm_device.h"

namespace ftmoe {

namespace {

template <typename E>
struct Piece {
  typedef E elems __attribute__((ext_vector_type(8)));
  typedef elems __attribute__((aligned(1))) any;
  elems v;
  __device__ __attribute__((always_inline)) inline void load(const E* p) { v = gload<any>(p); }
  __device__ __attribute__((always_inline)) inline void store(E* p) const { gstore<any>(p, v); }
};

// First column of a piece, and how many of its columns the one before has (8 or more: all).
struct Place {
  int c, skip;
  __device__ __attribute__((always_inline)) inline Place(int piece, int cols) {
    c = min(8 * piece, cols - 8);
    skip = 8 * piece - c;
  }
  __device__ __attribute__((always_inline)) inline bool some() const { return skip < 8; }
};

template <typename X, typename R, int THREADS, int PIECES>
__global__ __launch_bounds__(THREADS) void k_norm(NormForward a) {
  __shared__ double lds[3 * (THREADS / 64)];
  const X* weight = static_cast<const X*>(a.weight);
  const int64_t row = int64_t(blockIdx.y) * kNormGrid + blockIdx.x;
  if (row >= a.rows) return;
  const X* x = static_cast<const X*>(a.x) + row * a.ld_x;
  const R* residual = static_cast<const R*>(a.residual) + row * a.ld_residual;
  Piece<X> xv[PIECES], wv[PIECES];
  Piece<R> rv[PIECES];
#pragma unroll
  for (int g = 0; g < PIECES; ++g) {
    const Place p(int(threadIdx.x) + g * THREADS, a.cols);
    xv[g].load(x + p.c);
    if (a.residual) rv[g].load(residual + p.c);
    else rv[g].v = typename Piece<R>::elems{};
  }
#pragma unroll
  for (int g = 0; g < PIECES; ++g) wv[g].load(weight + Place(int(threadIdx.x) + g * THREADS, a.cols).c);
  NormSums t;
#pragma unroll
  for (int g = 0; g < PIECES; ++g) {
    const Place p(int(threadIdx.x) + g * THREADS, a.cols);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const double s = double(float(xv[g].v[i])) + double(float(rv[g].v[i]));
      t.add(i >= p.skip ? s : 0.0, double(float(wv[g].v[i])));
    }
  }
  t.join<THREADS>(lds);
  const NormRow r(t, a.cols, a.eps);
  if (a.codes && threadIdx.x == 0) a.scale[row] = r.scale;
#pragma unroll
  for (int g = 0; g < PIECES; ++g) {
    const Place p(int(threadIdx.x) + g * THREADS, a.cols);
    if (!p.some()) continue;
    Piece<R> sum;
    Piece<X> y;
    double sw[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const double s = double(float(xv[g].v[i])) + double(float(rv[g].v[i]));
      sum.v[i] = R(float(s));
      sw[i] = s * double(float(wv[g].v[i]));
      y.v[i] = X(float(sw[i] * r.r));
    }
    if (a.sum) sum.store(static_cast<R*>(a.sum) + row * a.ld_sum + p.c);
    if (a.y) y.store(static_cast<X*>(a.y) + row * a.ld_y + p.c);
    if (a.codes) {
      typedef uint32_t words __attribute__((ext_vector_type(2)));
      typedef words __attribute__((aligned(1))) any;
      words w{};
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i / 4] |= uint32_t(r.code(sw[i]) & 0xFF) << (i % 4 * 8);
      gstore<any>(a.codes + row * a.ld_codes + p.c, w);
    }
  }
}

// Rows blockIdx.x, + groups, ...; each thread sums its columns' weight gradients over them.
template <typename X, typename R, int THREADS, int PIECES, bool FAR>
__global__ __launch_bounds__(THREADS) void k_norm_backward(NormBackward a) {
  __shared__ double lds[2 * (THREADS / 64)];
  const X* weight = static_cast<const X*>(a.weight);
  float dw[PIECES][8] = {};
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    Piece<X> yv[PIECES], wv[PIECES];
    Piece<R> sv[PIECES], dv[PIECES];
#pragma unroll
    for (int g = 0; g < PIECES; ++g) {
      const int c = Place(int(threadIdx.x) + g * THREADS, a.cols).c;
      sv[g].load(static_cast<const R*>(a.sum) + row * a.ld_sum + c);
      yv[g].load(static_cast<const X*>(a.dy) + row * a.ld_y + c);
      wv[g].load(weight + c);
    }
#pragma unroll
    for (int g = 0; g < PIECES; ++g) {
      const int c = Place(int(threadIdx.x) + g * THREADS, a.cols).c;
      if (a.dsum) dv[g].load(static_cast<const R*>(a.dsum) + row * a.ld_residual + c);
      else dv[g].v = typename Piece<R>::elems{};
    }
    NormDots t;
#pragma unroll
    for (int g = 0; g < PIECES; ++g) {
      const Place p(int(threadIdx.x) + g * THREADS, a.cols);
      auto add = [&](int i) { t.add(float(sv[g].v[i]), float(yv[g].v[i]) * float(wv[g].v[i])); };
      if (p.skip == 0) {
#pragma unroll
        for (int i = 0; i < 8; ++i) add(i);
      } else {  // the row's last piece: left out, not taken as 0, which an infinity in dy would make a NaN
#pragma unroll
        for (int i = 0; i < 8; ++i)
          if (i >= p.skip) add(i);
      }
    }
    if (THREADS > 64 && row != blockIdx.x) __syncthreads();  // the last row's sums have been read
    t.join<THREADS>(lds);
    const NormSlope<FAR> k(t, a.cols, a.eps);
#pragma unroll
    for (int g = 0; g < PIECES; ++g) {
      const Place p(int(threadIdx.x) + g * THREADS, a.cols);
      if (!p.some()) continue;
      Piece<X> dx;
      Piece<R> dr;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float dy = float(yv[g].v[i]), n = k.n(float(sv[g].v[i]));
        const float ds = k.ds(dy * float(wv[g].v[i]), n) + float(dv[g].v[i]);
        dw[g][i] = fmaf(dy, n, dw[g][i]);
        dx.v[i] = X(ds);
        dr.v[i] = R(ds);
      }
      if (a.dx) dx.store(static_cast<X*>(a.dx) + row * a.ld_x + p.c);
      if (a.dresidual) dr.store(static_cast<R*>(a.dresidual) + row * a.ld_residual + p.c);
    }
  }
  if (!a.part && !a.dweight) return;
#pragma unroll
  for (int g = 0; g < PIECES; ++g) {
    const Place p(int(threadIdx.x) + g * THREADS, a.cols);
    if (!p.some()) continue;
    if (a.dweight) {
      Piece<X> v;
#pragma unroll
      for (int i = 0; i < 8; ++i) v.v[i] = X(dw[g][i]);
      v.store(static_cast<X*>(a.dweight) + p.c);
      continue;
    }
    Piece<float> v;
#pragma unroll
    for (int i = 0; i < 8; ++i) v.v[i] = dw[g][i];
    v.store(a.part + int64_t(blockIdx.x) * norm_part_ld(a.cols) + p.c);
  }
}

template <typename X, typename R, int THREADS, int PIECES>
hipError_t launch(const NormForward& a, hipStream_t s) {
  hipLaunchKernelGGL((k_norm<X, R, THREADS, PIECES>), norm_grid(a.rows), dim3(THREADS), 0, s, a);
  return hipGetLastError();
}
template <typename X, typename R, int THREADS, int PIECES>
hipError_t launch(const NormBackward& a, hipStream_t s) {
  const dim3 grid(uint32_t(a.groups));
  if (a.eps > 0.0) hipLaunchKernelGGL((k_norm_backward<X, R, THREADS, PIECES, false>), grid, dim3(THREADS), 0, s, a);
  else hipLaunchKernelGGL((k_norm_backward<X, R, THREADS, PIECES, true>), grid, dim3(THREADS), 0, s, a);
  return hipGetLastError();
}

template <typename X, typename R, typename A>
hipError_t launch_width(const A& a, hipStream_t s) {
  // Threads for up to four pieces each, the fewer the better: 8192 rows of 7168, us, by 256 x 4 / 512 x 2 / 1024 x 1:
  // codes and y 107 / 109 / 147, gradients (32-bit stream) 182 / 185 / 188; 32 rows of 6144: 5.2 / 5.2 / 6.3; 8192 rows
  // of 4096 by 128 x 4 / 256 x 2 / 512 x 1: codes and y 61 / 59 / 70; of 2048 by 128 x 2 / 256 x 1: 33 / 38, gradients
  // 40 / 36.  Chosen on 16-bit rows; 32-bit ones run at a copy's rate or past it by the same table (8192 x 2048 / 8192 x
  // 4096 / 4096 x 7168, forward 51 / 99 / 89 us, with codes 56 / 108 / 97, gradients 52 / 105 / 96: 4.9 to 5.4 TB/s).
  if (a.cols <= 512) return launch<X, R, 64, 1>(a, s);
  if (a.cols <= 2048) return launch<X, R, 256, 1>(a, s);
  if (a.cols <= 4096) return launch<X, R, 256, 2>(a, s);
  if (a.cols <= 8192) return launch<X, R, 256, 4>(a, s);
  return launch<X, R, 512, 4>(a, s);
}

template <typename A>
hipError_t launch_types(int dtype, int residual_dtype, const A& a, hipStream_t s) {
  const bool same = dtype == residual_dtype;
  if (dtype == FT_DT_F32) return launch_width<float, float>(a, s);
  if (dtype == FT_DT_F16) return same ? launch_width<_Float16, _Float16>(a, s) : launch_width<_Float16, float>(a, s);
  return same ? launch_width<__bf16, __bf16>(a, s) : launch_width<__bf16, float>(a, s);
}

}  // namespace

bool norm_rows(int32_t cols) { return cols >= 8 && cols <= 16384; }

hipError_t launch_norm_rows(int dtype, int residual_dtype, const NormForward& a, hipStream_t s) {
  return launch_types(dtype, residual_dtype, a, s);
}
hipError_t launch_norm_rows(int dtype, int residual_dtype, const NormBackward& a, hipStream_t s) {
  return launch_types(dtype, residual_dtype, a, s);
}

}  // namespace ftmoe
