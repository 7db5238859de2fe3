// A row's 8-bit codes and scale: scale = fp32(max|x| / 127), code = x / scale
// rounded to the nearest integer, ties to even.
//
// The quotient is rounded correctly without a division: n = rint(x * r) with
// r about 1 / scale is within one of the result, and d = x - n * scale, which a
// fused multiply-add gives exactly (it is a multiple of the smaller unit in
// the last place of x and scale, and no larger than scale), says which
// neighbour is nearer and where a tie is.  So codes depend neither on the
// reciprocal's accuracy nor on the order in which a row is walked.  Only a
// piece that holds some |d| of half the scale or more looks closer; else n
// stands, and lies in the low byte of x * r + 1.5 * 2^23.
#pragma once
#include "dense.h"

namespace ftmoe {

// 16 bytes of a row
template <typename E>
struct RowPiece {
  static constexpr int N = 16 / int(sizeof(E));
  typedef E elems __attribute__((ext_vector_type(N)));
  elems v;
  // from column c, whole if it is there, else zeros
  __device__ __attribute__((always_inline)) inline void load(const E* x, int c, int cols) {
    typedef elems __attribute__((aligned(1))) any;
    v = elems{};
    if (c + N <= cols) v = gload<any>(x + c);
  }
  // the piece that the row ends in, with zeros behind.  One thread's work, and apart
  // from the above: code for single elements at each piece took longer to fetch than to run.
  __device__ __attribute__((always_inline)) inline void load_last(const E* x, int cols) {
    const int c = cols / N * N;
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = c + i < cols ? gload<E>(x + c + i) : E(0);
  }
};

// The largest magnitude: magnitudes compare as integers, infinities and NaN
// lie above every finite one.
template <typename E>
struct RowMax {
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  uint32_t top = 0;  // 16-bit types: of the even columns, and of the odd ones above
  __device__ __attribute__((always_inline)) inline void add(const RowPiece<E>& p) {
    const u32x4 b = (u32x4)p.v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(E) == 4) {
        top = max(top, b[i] & 0x7FFFFFFFu);
      } else {
        const uint32_t m = b[i] & 0x7FFF7FFFu;
        const u16x2 t = __builtin_elementwise_max(__builtin_bit_cast(u16x2, top), __builtin_bit_cast(u16x2, m));
        top = __builtin_bit_cast(uint32_t, t);
      }
    }
  }
  // as the bits of an fp32
  __device__ __attribute__((always_inline)) inline uint32_t bits() const {
    if constexpr (sizeof(E) == 4) {
      return top;
    } else {
      const uint16_t m = uint16_t(max(top & 0xFFFFu, top >> 16));
      return __float_as_uint(float(__builtin_bit_cast(E, m)));
    }
  }
};

struct RowScale {
  float scale;          // as it is stored
  float s, r, k;        // k * scale, its reciprocal; tiny scales are taken into the normal range, exactly, by k
  uint32_t live;        // all ones, or 0 where every code is 0
  bool tiny;
  __device__ __attribute__((always_inline)) inline explicit RowScale(uint32_t top) {
    const bool finite = top < 0x7F800000u;
    scale = finite ? __uint_as_float(top) / 127.0f : __uint_as_float(0x7FC00000u);
    const bool on = finite && scale > 0.f;
    live = on ? ~0u : 0u;
    tiny = scale < 0x1p-100f;
    k = tiny ? 0x1p100f : 1.0f;
    s = on ? scale * k : 1.0f;
    r = __builtin_amdgcn_rcpf(s);
  }
  __device__ __attribute__((always_inline)) inline uint32_t close(float x) const {
    x *= k;
    float n = rintf(x * r);
    const float d = fmaf(-n, s, x), half = 0.5f * s;
    const bool odd = (int(n) & 1) != 0;
    if (d > half || (d == half && odd)) n += 1.0f;
    if (d < -half || (d == -half && odd)) n -= 1.0f;
    return uint32_t(int(fminf(fmaxf(n, -127.0f), 127.0f)));
  }
  // four or eight codes, a byte each
  template <typename E>
  __device__ __attribute__((always_inline)) inline void codes(const RowPiece<E>& p, uint32_t (&out)[RowPiece<E>::N / 4]) const {
    constexpr int N = RowPiece<E>::N;
    constexpr float kUnits = 12582912.0f;  // 1.5 * 2^23: a sum's last bit is 1
    uint32_t q[N];
    float far = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float x = float(p.v[i]), t = fmaf(x, r, kUnits);
      far = fmaxf(far, fabsf(fmaf(-(t - kUnits), s, x)));
      q[i] = __float_as_uint(t);
    }
    if (tiny || far >= 0.5f * s) {
#pragma unroll
      for (int i = 0; i < N; ++i) q[i] = close(float(p.v[i]));
    }
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const uint32_t lo = __builtin_amdgcn_perm(q[4 * i + 1], q[4 * i], 0x0C0C0400u);
      const uint32_t hi = __builtin_amdgcn_perm(q[4 * i + 3], q[4 * i + 2], 0x0C0C0400u);
      out[i] = __builtin_amdgcn_perm(hi, lo, 0x05040100u) & live;
    }
  }
};

}  // namespace ftmoe
