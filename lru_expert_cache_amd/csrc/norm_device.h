// Sums of a row and what follows from them.
//
// Forward: with p = s * weight, y = p r, r = 1 / sqrt(mean(s^2) + eps).  A
// row's codes are rint(y / scale), and have to be those of the exact y: all of
// it is formed in 64 bits (s of 16-bit addends and p are then exact), which
// leaves one y in about 2^40 on the wrong side of a border between two codes,
// and costs little: the 64-bit units keep up with the memory.  s and y go to
// 16 bits by way of 32: the instructions that convert start from there, and what
// that second rounding turns the other way lies within 2^-24 of a tie.
//
// Backward: with n = s r and g = dy weight, ds = r (g - n mean(g n)); only the
// two sums are formed in 64 bits.
#pragma once
#include "norm.h"

namespace ftmoe {

// a workgroup for each row, as many across as any workgroup size allows
constexpr int32_t kNormGrid = 1 << 21;
inline dim3 norm_grid(int32_t rows) {
  return dim3(uint32_t(rows < kNormGrid ? rows : kNormGrid), uint32_t((rows + kNormGrid - 1) / kNormGrid));
}

__device__ __attribute__((always_inline)) inline double wave_add(double v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}
__device__ __attribute__((always_inline)) inline double wave_max(double v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = fmax(v, __shfl_xor(v, o));
  return v;
}

struct NormSums {
  double squares = 0.0, top = 0.0;
  double odd = 0.0;  // NaN once a weighted value is infinite or NaN: a maximum alone would pass over it
  __device__ __attribute__((always_inline)) inline void add(double s, double w) {
    const double p = s * w;
    squares = fma(s, s, squares);
    top = fmax(top, fabs(p));
    odd = fma(p, 0.0, odd);
  }
  // of all threads of the workgroup; lds: three numbers a wave
  template <int THREADS>
  __device__ __attribute__((always_inline)) inline void join(double* lds) {
    squares = wave_add(squares);
    top = wave_max(top);
    odd = wave_add(odd);
    if constexpr (THREADS > 64) {
      const int wave = threadIdx.x >> 6;
      if ((threadIdx.x & 63) == 0) {
        lds[3 * wave] = squares;
        lds[3 * wave + 1] = top;
        lds[3 * wave + 2] = odd;
      }
      __syncthreads();
      squares = top = odd = 0.0;
#pragma unroll
      for (int i = 0; i < THREADS / 64; ++i) {
        squares += lds[3 * i];
        top = fmax(top, lds[3 * i + 1]);
        odd += lds[3 * i + 2];
      }
    }
  }
};

struct NormRow {
  double r;       // y = p r
  float scale;
  double q;       // code = rint(p q)
  bool live;      // else every code is 0
  __device__ __attribute__((always_inline)) inline NormRow(const NormSums& t, int cols, double eps) {
    r = 1.0 / sqrt(t.squares / cols + eps);
    const double top = t.top * r + t.odd;
    const bool finite = top < __builtin_huge_val();  // not NaN either
    scale = finite ? float(top / 127.0) : __uint_as_float(0x7FC00000u);
    live = finite && scale > 0.f;
    q = live ? r / double(scale) : 0.0;
  }
  // scales of few bits (next to the smallest fp32) leave quotients beyond 127
  __device__ __attribute__((always_inline)) inline int code(double p) const {
    return live ? min(max(int(rint(p * q)), -127), 127) : 0;
  }
};

struct NormDots {
  double squares = 0.0, dot = 0.0;
  __device__ __attribute__((always_inline)) inline void add(float s, float g) {
    squares = fma(double(s), double(s), squares);
    dot = fma(double(s), double(g), dot);
  }
  template <int THREADS>
  __device__ __attribute__((always_inline)) inline void join(double* lds) {
    squares = wave_add(squares);
    dot = wave_add(dot);
    if constexpr (THREADS > 64) {
      const int wave = threadIdx.x >> 6;
      if ((threadIdx.x & 63) == 0) {
        lds[2 * wave] = squares;
        lds[2 * wave + 1] = dot;
      }
      __syncthreads();
      squares = dot = 0.0;
#pragma unroll
      for (int i = 0; i < THREADS / 64; ++i) {
        squares += lds[2 * i];
        dot += lds[2 * i + 1];
      }
    }
  }
};

// FAR, for an eps of 0: 1 / sqrt(mean(s^2)) as up r.  It then reaches from
// 2^-128 to 2^161, beyond 32 bits; up is a power of two, and 1 within 2^100
// either way.  (An eps above 0 is 2^-149 or more, and keeps it below 2^75.
// Both products always: 8192 rows of 2048, bf16, 37.9 us against 36.7.)
template <bool FAR>
struct NormSlope {
  float up = 1.f, r, m;  // of n = s up r: ds = up r (g - n m), m = mean(g n)
  __device__ __attribute__((always_inline)) inline NormSlope(float r_, float m_, float up_) : up(up_), r(r_), m(m_) {}
  __device__ __attribute__((always_inline)) inline NormSlope(const NormDots& t, int cols, double eps) {
    const double rr = 1.0 / sqrt(t.squares / cols + eps);
    r = float(rr);
    if constexpr (FAR) {
      const bool large = rr > 0x1p100, small = rr < 0x1p-100;
      up = large ? 0x1p100f : small ? 0x1p-100f : 1.f;
      r = float(rr * (large ? 0x1p-100 : small ? 0x1p100 : 1.0));
    }
    m = float(rr * (t.dot / cols));
  }
  __device__ __attribute__((always_inline)) inline float n(float s) const { return FAR ? s * up * r : s * r; }
  __device__ __attribute__((always_inline)) inline float ds(float g, float n) const {
    const float v = fmaf(-n, m, g);
    return FAR ? v * up * r : v * r;
  }
};

}  // namespace ftmoe
