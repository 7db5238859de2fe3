// Dense (not routed) feed-forward operators: what their translation units share.
//
// Every operator is made of matrix products of one form,
//   C[m][n] = sum_k A(m, k) B(n, k),   m a token or a weight row, n contiguous in C,
// whose operands lie in memory either along K ("K rows": element (r, k) at
// r * ld + k) or across it ("K columns": at k * ld + r):
//   forward  g, u = x Wg^T, x Wu^T     A = x   K rows      B = Wg, Wu  K rows      -> h (and gu)
//            y = h Wd^T                A = h   K rows      B = Wd      K rows
//   backward dh = dy Wd                A = dy  K rows      B = Wd      K columns   -> dg, du, h
//            dx = dg Wg + du Wu        A = dgu K rows      B = Wg, Wu  K columns   (two K segments)
//            dWg, dWu, dWd             A = dg, du, dy, K columns       B = x, x, h  K columns   (K = tokens)
//   8 bit    as forward, on codes, with the scales applied to the exact sums
// Products are given as DenseProblems; one launch takes up to three of the same form.
#pragma once
#include "common.h"
#include "gmem.h"

namespace ftmoe {

// How a product's operands lie and what becomes of its sums.
enum DenseForm {
  kDenseGated = 0,  // K rows x K rows, two B matrices: h = silu(g) * u, and gu when given
  kDenseRows,       // K rows x K rows: c = sums
  kDenseGrad,       // K rows x K columns: sums are dh; reads gu, writes dgu, and h unless c is null
  kDenseCols,       // K rows x K columns: c = sums, one or two K segments
  kDenseOuter,      // K columns x K columns: c = sums
  kDenseInt,        // 8-bit codes, K rows x K rows: c = xs[m] ws[n] sums
  kDenseIntGated,   // 8-bit codes, two B matrices: h in fp32
  kDenseForms
};
constexpr bool dense_a_rows(int form) { return form != kDenseOuter; }
constexpr bool dense_b_rows(int form) {
  return form == kDenseGated || form == kDenseRows || form == kDenseInt || form == kDenseIntGated;
}
constexpr bool dense_two_b(int form) { return form == kDenseGated || form == kDenseIntGated; }
constexpr int dense_elem(int form) { return form == kDenseInt || form == kDenseIntGated ? 1 : 2; }
constexpr bool dense_int(int form) { return form == kDenseInt || form == kDenseIntGated; }

struct DenseProblem {
  const uint8_t* a[2];   // by K segment
  const uint8_t* b[2];   // by K segment (kDenseCols), or the two matrices of a gated form
  int64_t lda, ldb;      // bytes
  int32_t m, n, k;       // k: elements of each K segment
  int32_t segs;          // K segments, 1 or 2
  uint8_t* c;            // h for the gated forms and kDenseGrad
  int64_t ldc;           // elements, as the following
  uint8_t* gu;           // kDenseGated: written unless null; kDenseGrad: read
  int64_t ldgu, off_u;   // u's first column in gu
  uint8_t* dgu;          // kDenseGrad: written
  int64_t lddgu, off_du;
  int32_t c_lo;          // kDenseGated, kDenseGrad: rows from a rounded h, dg, du to what its rounding left off; 0: not kept
  int32_t a_lo;          // rows from A's values to what their rounding left off, which is added; 0: A has one part
  const float* xs;       // 8-bit forms: scale per row, per column (of each matrix)
  const float* ws[2];
  int32_t tokens;        // 8-bit forms, few tokens: a's type where it is yet to be quantised (kDenseInt: FT_DT_F32;
                         // kDenseIntGated: FT_DT_BF16, FT_DT_F16), else 0
  bool a_whole, b_whole; // this operand's rows are zeros up to a whole 16-byte piece
  uint8_t* part;         // split K: 32-bit sums [split][matrix][m][n rounded up to 4], else null
};
constexpr int kDenseMaxProblems = 3;
// h, dg and du are rounded to 16 bits for the next products.  Over many tokens
// and columns that adds up to 1.4 times the result's own rounding; with few it
// scatters (1 token, I 128 to 768: over 1.5 times for a quarter of the inputs,
// 2.6 at worst).  Up to these numbers of tokens the products take both 16-bit
// parts of such a value, in places that would stay empty: the forward pass in
// the second eight of a fragment's 16 rows (9 to 16 tokens: in a second
// fragment), dx in the second 64 of a tile's 128, the weight gradients in a
// second K step that the first is paired with anyway.
constexpr int kDenseLoForward = 16, kDenseLoBackward = 64;
// rows from a value to its rest
constexpr int dense_lo(int tokens, bool backward) {
  return tokens == 0 || tokens > (backward ? kDenseLoBackward : kDenseLoForward) ? 0 : backward ? 64 : tokens <= 8 ? 8 : 16;
}
struct DenseLaunch {
  DenseProblem p[kDenseMaxProblems];
  int32_t count;
  int32_t splits;        // parts that K is cut into (tiled kernels)
  int32_t tiles;         // of all problems (set by the launchers)
  uint32_t* clear;       // kDenseQueue counters that the tiled kernels set to zero, or null
};

// The backward pass's last products in one launch: the weight gradients
// (kDenseOuter, not cut into parts) and dx (kDenseCols) share the workgroups,
// which take tiles from one queue per XCD, the longer ones (the weight
// gradients') first.  The queue counters must be zero at the start: the launch
// before, of dh, clears them.  Which workgroup takes a tile changes no result.
constexpr int kDenseQueue = 8;
struct DensePair {
  DenseLaunch outer, cols;
  uint32_t* queue;
};

// How a product (or up to three of one form) is run on the tiled kernels:
// 256 x 256 or 128 x 128 tiles, K cut into `splits` parts whose sums are then
// added in order by a second kernel.  A rule on sizes alone (dense_plan.cpp).
struct DensePlan {
  int32_t tile;
  int32_t splits;
};
struct DenseShape {
  int32_t m, n, k, segs;
};
DensePlan dense_plan(DenseForm form, const DenseShape* shapes, int count);
// the tile of a DensePair, or 0 where separate launches are quicker; only128: 256 x 256 is not there for it
int dense_plan_pair(const DenseShape (&outer)[3], const DenseShape& cols, bool only128 = false);
int64_t dense_part_bytes(DenseForm form, const DenseShape& s, int splits);

// dense_any.hip: any size, stride and alignment.  dtype: FT_DT_* of the
// operands (16-bit forms) or of c (kDenseInt).
hipError_t launch_dense_any(DenseForm form, int dtype, const DenseLaunch& l, hipStream_t s);

// dense_tile_*.hip: operands on 16-byte addresses and row distances (dense_tileable)
bool dense_tileable(DenseForm form, const DenseProblem& p);
hipError_t launch_dense_tile(DenseForm form, int dtype, int tile, const DenseLaunch& l, hipStream_t s);
hipError_t launch_dense_tile_bf16(DenseForm form, int tile, const DenseLaunch& l, hipStream_t s);
hipError_t launch_dense_tile_f16(DenseForm form, int tile, const DenseLaunch& l, hipStream_t s);
hipError_t launch_dense_pair(int dtype, int tile, const DensePair& l, hipStream_t s);
hipError_t launch_dense_pair_bf16(int tile, const DensePair& l, hipStream_t s);
hipError_t launch_dense_pair_f16(int tile, const DensePair& l, hipStream_t s);
hipError_t launch_dense_tile_int(DenseForm form, int dtype, int tile, const DenseLaunch& l, hipStream_t s);

// dense_few.hip: tileable products of up to kDenseFewRows tokens, both operands along K
constexpr int kDenseFewRows = 64;
// 8-bit forms: whether it can quantise m tokens of k elements itself
bool dense_few_quantizes(int m, int k);
hipError_t launch_dense_few(DenseForm form, int dtype, const DenseLaunch& l, hipStream_t s);

// dense_pack.hip: rows of `bytes` bytes copied to dst rows of dst_bytes (a
// multiple of 16, at 16-byte addresses), zeros behind them; src is not read when bytes is 0
struct DensePack {
  const uint8_t* src;
  uint8_t* dst;
  int64_t src_ld, dst_ld, bytes, dst_bytes, rows;
  int32_t lanes;  // set by the launch
};
constexpr int kDenseMaxPacks = 8;  // a backward pass: x, dy, three weights, h, dg, du
struct DensePackLaunch {
  DensePack p[kDenseMaxPacks];
  int32_t count;
};
hipError_t launch_dense_pack(const DensePackLaunch& l, hipStream_t s);

// int_quant.hip: rows of x (FT_DT_*) to 8-bit codes and scales
hipError_t launch_int_quantize(int dtype, int32_t rows, int32_t cols, const void* x, int64_t ld_x, int8_t* codes,
                               int64_t ld_codes, float* scale, hipStream_t s);

#ifdef __HIPCC__
// ------------------------------------------------------------ device side
typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef float floatx16 __attribute__((ext_vector_type(16)));
typedef int intx4 __attribute__((ext_vector_type(4)));
typedef int intx16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef _Float16 f16x4 __attribute__((ext_vector_type(4)));

// Operand types.  A 16x16 matrix instruction takes 16 bytes of K per lane of
// either operand: lane l holds row l % 16, K bytes 16 (l / 16) .. + 15 of a
// 64-byte step, and the sums of first-operand rows 4 (l / 16) + i and
// second-operand row l % 16, i = 0..3.  A 32x32 matrix instruction takes 16 bytes of K per lane of
// either operand: lane l holds row l % 32, K bytes 16 (l / 32) .. + 15 of a
// 32-byte step, and the sums of first-operand rows 8 (i / 4) + 4 (l / 32) +
// i % 4 and second-operand row l % 32.
struct DenseBf16 {
  typedef __bf16 elem;
  typedef bf16x4 elem4;
  typedef floatx16 acc;
  typedef float sum;
  static __device__ __attribute__((always_inline)) inline acc mfma(u32x4 a, u32x4 b, acc c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_bf16((bf16x8)a, (bf16x8)b, c, 0, 0, 0);
  }
  typedef floatx4 acc4;
  static __device__ __attribute__((always_inline)) inline acc4 mfma16(u32x4 a, u32x4 b, acc4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16((bf16x8)a, (bf16x8)b, c, 0, 0, 0);
  }
};
struct DenseF16 {
  typedef _Float16 elem;
  typedef f16x4 elem4;
  typedef floatx16 acc;
  typedef float sum;
  static __device__ __attribute__((always_inline)) inline acc mfma(u32x4 a, u32x4 b, acc c) {
    return __builtin_amdgcn_mfma_f32_32x32x16_f16((f16x8)a, (f16x8)b, c, 0, 0, 0);
  }
  typedef floatx4 acc4;
  static __device__ __attribute__((always_inline)) inline acc4 mfma16(u32x4 a, u32x4 b, acc4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16((f16x8)a, (f16x8)b, c, 0, 0, 0);
  }
};
struct DenseI8 {
  typedef int8_t elem;
  typedef intx16 acc;
  typedef int sum;
  static __device__ __attribute__((always_inline)) inline acc mfma(u32x4 a, u32x4 b, acc c) {
    return __builtin_amdgcn_mfma_i32_32x32x32_i8((intx4)a, (intx4)b, c, 0, 0, 0);
  }
  typedef intx4 acc4;
  static __device__ __attribute__((always_inline)) inline acc4 mfma16(u32x4 a, u32x4 b, acc4 c) {
    return __builtin_amdgcn_mfma_i32_16x16x64_i8((intx4)a, (intx4)b, c, 0, 0, 0);
  }
};

// 1 / (1 + e^-g) from the hardware exp2 and reciprocal (each about 1 ulp);
// e^-g overflowing to infinity gives 0
__device__ inline float dense_sigmoid(float g) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -1.4426950408889634f));
}

// N neighbouring elements of a row at once, whatever their alignment (the
// memory system takes any), or the cnt that exist one by one
template <typename E, int N>
struct DenseRun {
  typedef E plain __attribute__((ext_vector_type(N)));
  typedef plain __attribute__((aligned(1))) any;
};
template <typename E, int N>
__device__ __attribute__((always_inline)) inline void dense_store(uint8_t* base, int64_t at, const float* v, int cnt) {
  E* p = reinterpret_cast<E*>(base) + at;
  if (cnt == N) {
    typename DenseRun<E, N>::plain x;
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = E(v[i]);
    gstore<typename DenseRun<E, N>::any>(p, x);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (i < cnt) gstore<E>(p + i, E(v[i]));
  }
}

// What the sums of row m, columns n .. n + cnt - 1 are combined with, read
// ahead of the stores (which the compiler cannot move reads across).
template <int FORM, typename E, int N>
struct DenseWith {};
template <typename E, int N>
struct DenseWith<kDenseGrad, E, N> {
  typename DenseRun<E, N>::plain g, u;
  // from a place that exists, whole
  __device__ __attribute__((always_inline)) inline void fetch(const DenseProblem& p, int64_t m, int n) {
    const E* s = reinterpret_cast<const E*>(p.gu) + m * p.ldgu + n;
    g = gload<typename DenseRun<E, N>::any>(s);
    u = gload<typename DenseRun<E, N>::any>(s + p.off_u);
  }
  __device__ __attribute__((always_inline)) inline void fetch(const DenseProblem& p, int64_t m, int n, int cnt) {
    const E* s = reinterpret_cast<const E*>(p.gu) + m * p.ldgu + n;
    if (cnt == N) {
      g = gload<typename DenseRun<E, N>::any>(s);
      u = gload<typename DenseRun<E, N>::any>(s + p.off_u);
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) {
        g[i] = i < cnt ? gload<E>(s + i) : E(0);
        u[i] = i < cnt ? gload<E>(s + p.off_u + i) : E(0);
      }
    }
  }
};
// scales of N columns (of each matrix)
template <int N>
struct DenseScales {
  float w0[N], w1[N];
  template <bool TWO>
  __device__ __attribute__((always_inline)) inline void fetch(const DenseProblem& p, int n) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int at = n + i < p.n ? n + i : p.n - 1;
      w0[i] = gload<float>(p.ws[0] + at);
      w1[i] = TWO ? gload<float>(p.ws[1] + at) : 0.f;
    }
  }
};

// What becomes of the sums of row m, columns n .. n + cnt - 1 (cnt <= N); v1: the second matrix of a gated form.  E: the operands'
// type, TO: c's type where it differs (8-bit forms).  Rounding: h, g, u, dg
// and du are rounded once, to the type they are stored in, from fp32 values.
// That of h, dg and du is chosen: the next product's matrix instructions take
// 16-bit operands at 16 times fp32's rate, and half the bytes come back.  It
// costs the result 1.4 times the error of rounding it alone (relative 2-norm
// 0.0024 in bf16, 0.0017 without), and in fp16 the range beyond 65504; few
// tokens keep what it left off (kDenseLoForward).
// LO: what the rounding of h, dg and du left off is stored too where c_lo asks
// for it.
// (the rest, rounded to E; 0 beside infinities and NaN)
template <typename E, int N>
__device__ __attribute__((always_inline)) inline void dense_store_rest(uint8_t* base, int64_t at, const float* v, int cnt) {
  float r[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const float hi = float(E(v[i]));
    r[i] = __builtin_isfinite(hi) ? v[i] - hi : 0.0f;
  }
  dense_store<E, N>(base, at, r, cnt);
}
template <int FORM, typename E, typename TO, int N, bool LO>
__device__ __attribute__((always_inline)) inline void dense_emit(const DenseProblem& p, int64_t m, int n, int cnt,
                                                                 const float* v0, const float* v1,
                                                                 const DenseWith<FORM, E, N>& with) {
  if constexpr (FORM == kDenseRows || FORM == kDenseCols || FORM == kDenseOuter) {
    dense_store<TO, N>(p.c, m * p.ldc + n, v0, cnt);
  } else if constexpr (FORM == kDenseGated) {
    float h[N];
#pragma unroll
    for (int i = 0; i < N; ++i) h[i] = v0[i] * dense_sigmoid(v0[i]) * v1[i];
    dense_store<TO, N>(p.c, m * p.ldc + n, h, cnt);
    if (LO && p.c_lo) dense_store_rest<TO, N>(p.c, (m + p.c_lo) * p.ldc + n, h, cnt);
    if (p.gu) {
      dense_store<TO, N>(p.gu, m * p.ldgu + n, v0, cnt);
      dense_store<TO, N>(p.gu, m * p.ldgu + p.off_u + n, v1, cnt);
    }
  } else {
    static_assert(FORM == kDenseGrad, "8-bit sums take their scales");
    float dg[N], du[N], h[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float g = float(with.g[i]), u = float(with.u[i]);
      const float s = dense_sigmoid(g), gs = g * s;
      dg[i] = v0[i] * u * s * (1.0f + g * (1.0f - s));
      du[i] = v0[i] * gs;
      h[i] = gs * u;
    }
    dense_store<E, N>(p.dgu, m * p.lddgu + n, dg, cnt);
    dense_store<E, N>(p.dgu, m * p.lddgu + p.off_du + n, du, cnt);
    if (p.c) dense_store<E, N>(p.c, m * p.ldc + n, h, cnt);
    if (LO && p.c_lo) {
      dense_store_rest<E, N>(p.dgu, (m + p.c_lo) * p.lddgu + n, dg, cnt);
      dense_store_rest<E, N>(p.dgu, (m + p.c_lo) * p.lddgu + p.off_du + n, du, cnt);
      if (p.c) dense_store_rest<E, N>(p.c, (m + p.c_lo) * p.ldc + n, h, cnt);
    }
  }
}
// the 8-bit forms: the int32 sums are exact; their conversion and the scales round in fp32
template <int FORM, typename TO, int N>
__device__ __attribute__((always_inline)) inline void dense_emit(const DenseProblem& p, int64_t m, int n, int cnt,
                                                                 const int* v0, const int* v1, float xs,
                                                                 const DenseScales<N>& ws) {
  float v[N];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    v[i] = float(v0[i]) * xs * ws.w0[i];
    if constexpr (FORM == kDenseIntGated) v[i] = v[i] * dense_sigmoid(v[i]) * (float(v1[i]) * xs * ws.w1[i]);
  }
  dense_store<TO, N>(p.c, m * p.ldc + n, v, cnt);
}
// the same with everything read on the spot
template <int FORM, typename E, typename TO, typename S>
__device__ __attribute__((always_inline)) inline void dense_finish(const DenseProblem& p, int64_t m, int n, int cnt,
                                                                   const S* v0, const S* v1) {
  if constexpr (dense_int(FORM)) {
    DenseScales<4> ws;
    ws.fetch<dense_two_b(FORM)>(p, n);
    dense_emit<FORM, TO, 4>(p, m, n, cnt, v0, v1, gload<float>(p.xs + m), ws);
  } else {
    DenseWith<FORM, E, 4> with;
    if constexpr (FORM == kDenseGrad) with.fetch(p, m, n, cnt);
    dense_emit<FORM, E, TO, 4, true>(p, m, n, cnt, v0, v1, with);
  }
}
#endif

}  // namespace ftmoe
