// The dense products for operands of any size, stride and alignment.
//
// A workgroup of four waves owns 64 x 64 results; each wave one 32 x 32
// quadrant (of both matrices in a gated form).  64 bytes of K per step are
// read in 16-byte pieces (an unaligned 16-byte global load where the piece is
// whole, single elements at an edge, zeros outside) into registers while the
// step before is multiplied, and stored to LDS along K, rows 80 bytes apart
// (16-byte reads of 8 neighbouring rows then fall into different banks).
// Operands that lie across K are turned while they are stored.
//
// Bound by the loads' and LDS stores' instruction count, not by the matrix
// cores: this kernel runs only what the tiled kernels cannot take.
#include "dense.h"

namespace ftmoe {

namespace {

constexpr int kTile = 64;     // rows and columns of a workgroup
constexpr int kStep = 64;     // bytes of K per step
constexpr int kPitch = 80;    // bytes between LDS rows

// One operand's 64-row piece of a K step, 16 bytes per thread.
template <typename E, bool ROWS>
struct AnyPiece {
  static constexpr int EP = 16 / int(sizeof(E));     // elements of a piece
  static constexpr int KS = kStep / int(sizeof(E));  // K elements of a step
  u32x4 v;

  __device__ inline void load(const uint8_t* base, int64_t ld, int64_t r0, int rows, int k0, int k) {
    const int tid = threadIdx.x;
    int64_t at;   // bytes
    int have;     // elements of the piece that exist
    if constexpr (ROWS) {
      const int r = tid >> 2, kk = k0 + (tid & 3) * EP;
      have = r0 + r < rows ? k - kk : 0;
      at = (r0 + r) * ld + int64_t(kk) * int64_t(sizeof(E));
    } else {
      const int kk = k0 + tid / (kTile / EP), r = (tid % (kTile / EP)) * EP;
      have = kk < k && kk < k0 + KS ? int(rows - r0 - r < EP ? rows - r0 - r : EP) : 0;
      at = int64_t(kk) * ld + (r0 + r) * int64_t(sizeof(E));
    }
    v = u32x4{0, 0, 0, 0};
    if (have >= EP) {
      typedef u32x4 __attribute__((aligned(1))) u32x4_any;
      v = gload<u32x4_any>(base + at);
    } else {
      E e[EP];
#pragma unroll
      for (int i = 0; i < EP; ++i) e[i] = i < have ? gload<E>(base + at + i * int(sizeof(E))) : E(0);
      __builtin_memcpy(&v, e, 16);
    }
  }
  __device__ inline void store(uint8_t* lds) const {
    const int tid = threadIdx.x;
    if constexpr (ROWS) {
      *reinterpret_cast<u32x4*>(lds + (tid >> 2) * kPitch + (tid & 3) * 16) = v;
    } else {
      const int kk = tid / (kTile / EP), r = (tid % (kTile / EP)) * EP;
      if (kk < KS) {
        E e[EP];
        __builtin_memcpy(e, &v, 16);
#pragma unroll
        for (int i = 0; i < EP; ++i) *reinterpret_cast<E*>(lds + (r + i) * kPitch + kk * int(sizeof(E))) = e[i];
      }
    }
  }
};

template <typename D, int FORM, typename TO>
__global__ __launch_bounds__(256) void k_dense_any(DenseLaunch l) {
  typedef typename D::elem E;
  constexpr bool AR = dense_a_rows(FORM), BR = dense_b_rows(FORM);
  constexpr int NB = dense_two_b(FORM) ? 2 : 1;
  constexpr int KS = kStep / int(sizeof(E));
  __shared__ __attribute__((aligned(16))) uint8_t sa[kTile * kPitch];
  __shared__ __attribute__((aligned(16))) uint8_t sb[NB][kTile * kPitch];

  int64_t item = blockIdx.x;
  int pi = 0;
  for (;; ++pi) {  // uniform: the problem this workgroup belongs to
    const int64_t tiles = int64_t((l.p[pi].m + kTile - 1) / kTile) * ((l.p[pi].n + kTile - 1) / kTile);
    if (item < tiles || pi == l.count - 1) break;
    item -= tiles;
  }
  const DenseProblem& p = l.p[pi];
  const int tn = (p.n + kTile - 1) / kTile;
  const int64_t m0 = item / tn * kTile;
  const int n0 = int(item % tn) * kTile;
  if (m0 >= p.m) return;

  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
  const int mh = (w & 1) * 32, nh = (w >> 1) * 32;
  typename D::acc acc[NB];
#pragma unroll
  for (int j = 0; j < NB; ++j)
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[j][i] = 0;

  // K segments of A's values, then of what their rounding left off
  const int per = (p.k + KS - 1) / KS, steps = per * p.segs * (p.a_lo ? 2 : 1);
  AnyPiece<E, AR> pa;
  AnyPiece<E, BR> pb[NB];
  auto load = [&](int step) {
    const int at = step / per, lo = at >= p.segs, seg = at - lo * p.segs, k0 = (step - at * per) * KS;
    pa.load(p.a[seg] + (lo ? p.a_lo * p.lda : 0), p.lda, m0, p.m, k0, p.k);
#pragma unroll
    for (int j = 0; j < NB; ++j) pb[j].load(p.b[NB == 2 ? j : seg], p.ldb, n0, p.n, k0, p.k);
  };
  if (steps > 0) load(0);
  for (int step = 0; step < steps; ++step) {
    __syncthreads();  // the step before has been read
    pa.store(sa);
#pragma unroll
    for (int j = 0; j < NB; ++j) pb[j].store(sb[j]);
    __syncthreads();
    if (step + 1 < steps) load(step + 1);
#pragma unroll
    for (int q = 0; q < kStep / 32; ++q) {
      const int kb = q * 32 + (lane >> 5) * 16;
      const u32x4 a = *reinterpret_cast<const u32x4*>(sa + (mh + (lane & 31)) * kPitch + kb);
#pragma unroll
      for (int j = 0; j < NB; ++j) {
        const u32x4 b = *reinterpret_cast<const u32x4*>(sb[j] + (nh + (lane & 31)) * kPitch + kb);
        acc[j] = D::mfma(b, a, acc[j]);
      }
    }
  }

  const int64_t m = m0 + mh + (lane & 31);
  if (m >= p.m) return;
#pragma unroll
  for (int i = 0; i < 16; i += 4) {
    const int n = n0 + nh + 2 * i + (lane >> 5) * 4;
    typename D::sum v0[4], v1[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) v0[j] = acc[0][i + j], v1[j] = acc[NB - 1][i + j];
    const int cnt = p.n - n < 4 ? p.n - n : 4;
    if (cnt > 0) dense_finish<FORM, E, TO>(p, m, n, cnt, v0, v1);
  }
}

template <typename D, int FORM, typename TO>
hipError_t launch(const DenseLaunch& l, hipStream_t s) {
  int64_t tiles = 0;
  for (int i = 0; i < l.count; ++i)
    tiles += int64_t((l.p[i].m + kTile - 1) / kTile) * ((l.p[i].n + kTile - 1) / kTile);
  if (tiles == 0) return hipSuccess;
  if (tiles > INT32_MAX) return hipErrorInvalidValue;
  hipLaunchKernelGGL((k_dense_any<D, FORM, TO>), dim3(uint32_t(tiles)), dim3(256), 0, s, l);
  return hipGetLastError();
}

template <typename D>
hipError_t launch16(DenseForm form, const DenseLaunch& l, hipStream_t s) {
  typedef typename D::elem E;
  switch (form) {
    case kDenseGated: return launch<D, kDenseGated, E>(l, s);
    case kDenseRows: return launch<D, kDenseRows, E>(l, s);
    case kDenseGrad: return launch<D, kDenseGrad, E>(l, s);
    case kDenseCols: return launch<D, kDenseCols, E>(l, s);
    case kDenseOuter: return launch<D, kDenseOuter, E>(l, s);
    default: return hipErrorInvalidValue;
  }
}

}  // namespace

hipError_t launch_dense_any(DenseForm form, int dtype, const DenseLaunch& l, hipStream_t s) {
  if (form == kDenseIntGated) return launch<DenseI8, kDenseIntGated, float>(l, s);
  if (form == kDenseInt) {
    if (dtype == FT_DT_F32) return launch<DenseI8, kDenseInt, float>(l, s);
    if (dtype == FT_DT_F16) return launch<DenseI8, kDenseInt, _Float16>(l, s);
    return launch<DenseI8, kDenseInt, __bf16>(l, s);
  }
  return dtype == FT_DT_F16 ? launch16<DenseF16>(form, l, s) : launch16<DenseBf16>(form, l, s);
}

}  // namespace ftmoe
