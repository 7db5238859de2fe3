// Adapters: the second product, y = base + scale B h.
//
// h is the matrix instructions' second operand, in 16-bit parts that add up to
// its 32 bits: bf16 takes two for a 16-bit y (which keeps 16 bits of h: 2^-18
// off, against y's own 2^-9) and three for a 32-bit one, fp16 two (22 bits),
// with each token's row brought into fp16's range by a power of two.  Up to
// rank 16, two parts are one instruction of 32 ranks.
#include "adapters_device.h"

namespace ftmoe {

namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;

// KS: steps of 32 ranks; 0: up to 16 ranks, two parts in a step
template <typename D, typename B, typename Y, int SUB, int KS>
__global__ __launch_bounds__(kThreads) void k_adapters_out(Adapters l) {
  typedef typename D::elem E;
  typedef E elem8 __attribute__((ext_vector_type(8)));
  typedef float float8 __attribute__((ext_vector_type(8)));
  typedef float8 __attribute__((aligned(4))) float8_any;
  typedef B base8 __attribute__((ext_vector_type(8)));
  constexpr bool kHalf = sizeof(E) == 2 && __is_same(E, _Float16);
  constexpr int kParts = !kHalf && sizeof(Y) == 4 ? 3 : 2;
  constexpr int kSteps = KS == 0 ? 1 : KS;                              // of B's pieces
  constexpr int kFrags = KS == 0 ? (kParts + 1) / 2 : KS * kParts;      // of h's
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, q = lane >> 4;
  const int across = (l.out + 128 * l.out_blocks - 1) / (128 * l.out_blocks);
  const int64_t total = int64_t(l.windows) * l.tile_cap * across;
  for (int64_t flat = blockIdx.x; flat < total; flat += gridDim.x) {
    const TileTokens<SUB> t = find_tile<SUB>(l, flat / across);
    if (!t.live) continue;
    const int n0 = int(flat % across) * 128 * l.out_blocks + 32 * wave;
    const int n1 = int(min(int64_t(l.out), int64_t(flat % across + 1) * 128 * l.out_blocks));
    const bool on = t.id != l.count;

    // this lane's token and ranks: 8 (q mod 2) .. for KS 0, else 32 step + 8 q ..
    u32x4 h[SUB][kFrags] = {};
    float scale[SUB];
    if (on) {
#pragma unroll
      for (int m = 0; m < SUB; ++m) {
        float v[kSteps][8];
        float top = 0.f;
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          const int c = KS == 0 ? (q & 1) : 4 * k + q;  // piece of eight ranks, as row_piece takes it of B
          const float* row = l.h + int64_t(t.token[m]) * l.ld_h;
          const int from = min(8 * c, max(l.rank - 8, 0));
#pragma unroll
          for (int i = 0; i < 8; ++i) v[k][i] = 0.f;
          if (8 * c < l.rank) {
            if (l.rank >= 8) {
              float8 sum{};
              for (int p = 0; p < l.parts; ++p) sum += gload<float8_any>(row + int64_t(p) * l.tokens * l.ld_h + from);
#pragma unroll
              for (int i = 0; i < 8; ++i) v[k][i] = from + i >= 8 * c ? sum[i] : 0.f;
            } else {
              for (int p = 0; p < l.parts; ++p) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                  if (i < l.rank) v[k][i] += gload<float>(row + int64_t(p) * l.tokens * l.ld_h + i);
              }
            }
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(v[k][i]));
        }
        scale[m] = l.scale ? gload<float>(l.scale + t.id) : 1.f;
        if constexpr (kHalf) {
          // the row's largest value to 2^13 .. 2^14
          top = fmaxf(top, __shfl_xor(top, 16));
          top = fmaxf(top, __shfl_xor(top, 32));
          const int e = top > 0.f && top < __builtin_huge_valf() ? 14 - __builtin_amdgcn_frexp_expf(top) : 0;
          scale[m] = __builtin_ldexpf(scale[m], -e);
#pragma unroll
          for (int k = 0; k < kSteps; ++k)
#pragma unroll
            for (int i = 0; i < 8; ++i) v[k][i] = __builtin_ldexpf(v[k][i], e);
        }
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          elem8 part[kParts];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            float left = v[k][i];
#pragma unroll
            for (int p = 0; p < kParts; ++p) {
              part[p][i] = E(left);
              const float is = float(part[p][i]);
              left = __builtin_isfinite(is) ? left - is : 0.f;
            }
          }
          if constexpr (KS == 0) {
            h[m][0] = q < 2 ? (u32x4)part[0] : (u32x4)part[1];
            if constexpr (kParts == 3) h[m][1] = q < 2 ? (u32x4)part[2] : u32x4{};
          } else {
#pragma unroll
            for (int p = 0; p < kParts; ++p) h[m][k * kParts + p] = (u32x4)part[p];
          }
        }
      }
    }

    // A step's 32 columns: two instructions, whose rows 4 a + i are columns 8 a + 4 j + i: lane (q, token) gets
    // columns 8 q .. 8 q + 7.
    u32x4 b[2][kSteps];
    base8 with[SUB];
    const int mine = 8 * ((lane & 15) >> 2) + (lane & 3);
    auto fetch = [&](int n) {
      if (on) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const E* row = static_cast<const E*>(l.b) + (int64_t(t.id) * l.out + min(n + mine + 4 * j, l.out - 1)) * l.ld_b;
#pragma unroll
          for (int k = 0; k < kSteps; ++k) b[j][k] = row_piece<E, false>(row, KS == 0 ? (q & 1) : 4 * k + q, l.rank);
        }
      }
      const int c = n + 8 * q;
      if (l.base) {
#pragma unroll
        for (int m = 0; m < SUB; ++m) {
          const B* row = static_cast<const B*>(l.base) + int64_t(t.token[m]) * l.ld_base;
          typedef base8 __attribute__((aligned(1))) any;
          if (c + 8 <= l.out) {
            with[m] = gload<any>(row + c);
          } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) with[m][i] = c + i < l.out ? gload<B>(row + c + i) : B(0);
          }
        }
      }
    };
    if (n0 < n1) fetch(n0);
    for (int n = n0; n < n1; n += 128) {
      u32x4 bn[2][kSteps];
      base8 wn[SUB];
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int k = 0; k < kSteps; ++k) bn[j][k] = b[j][k];
#pragma unroll
      for (int m = 0; m < SUB; ++m) wn[m] = with[m];
      if (n + 128 < n1) fetch(n + 128);
#pragma unroll
      for (int m = 0; m < SUB; ++m) {
        float v[8] = {};
        if (on) {
          floatx4 acc[2] = {};
#pragma unroll
          for (int f = 0; f < kFrags; ++f)
#pragma unroll
            for (int j = 0; j < 2; ++j) acc[j] = D::mfma16(bn[j][KS == 0 ? 0 : f / kParts], h[m][f], acc[j]);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] = acc[i >> 2][i & 3] * scale[m];
        }
        if (l.base) {
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] += float(wn[m][i]);
        }
        const int c = n + 8 * q;
        if (16 * m + (lane & 15) < t.count && c < l.out)
          dense_store<Y, 8>(static_cast<uint8_t*>(l.y), int64_t(t.token[m]) * l.ld_y + c, v, min(8, l.out - c));
      }
    }
  }
}

template <typename D, typename B, typename Y, int SUB, int KS>
hipError_t launch(const Adapters& l, hipStream_t s) {
  const int64_t across = (l.out + 128 * l.out_blocks - 1) / (128 * l.out_blocks);
  const int64_t total = int64_t(l.windows) * l.tile_cap * across;
  hipLaunchKernelGGL((k_adapters_out<D, B, Y, SUB, KS>), dim3(uint32_t(total < (1 << 22) ? total : (1 << 22))),
                     dim3(kThreads), 0, s, l);
  return hipGetLastError();
}
template <typename D, typename B, typename Y>
hipError_t launch_form(const Adapters& l, hipStream_t s) {
  const int ks = l.rank <= 16 ? 0 : (l.rank + 31) / 32;
  if (l.sub == 1) {
    if (ks == 0) return launch<D, B, Y, 1, 0>(l, s);
    if (ks == 1) return launch<D, B, Y, 1, 1>(l, s);
    if (ks == 2) return launch<D, B, Y, 1, 2>(l, s);
    if (ks <= 4) return launch<D, B, Y, 1, 4>(l, s);
    return launch<D, B, Y, 1, 8>(l, s);
  }
  if (l.sub == 2) {
    if (ks == 0) return launch<D, B, Y, 2, 0>(l, s);
    if (ks == 1) return launch<D, B, Y, 2, 1>(l, s);
    return launch<D, B, Y, 2, 2>(l, s);
  }
  if (ks == 0) return launch<D, B, Y, 4, 0>(l, s);
  if (ks == 1) return launch<D, B, Y, 4, 1>(l, s);
  return launch<D, B, Y, 4, 2>(l, s);
}
template <typename D>
hipError_t launch_types(int base_dtype, int out_dtype, const Adapters& l, hipStream_t s) {
  typedef typename D::elem E;
  if (out_dtype == FT_DT_F32) return launch_form<D, float, float>(l, s);
  if (base_dtype == FT_DT_F32) return launch_form<D, float, E>(l, s);
  return launch_form<D, E, E>(l, s);
}

}  // namespace

hipError_t launch_adapters_out(int dtype, int base_dtype, int out_dtype, const Adapters& l, hipStream_t s) {
  return dtype == FT_DT_F16 ? launch_types<DenseF16>(base_dtype, out_dtype, l, s)
                            : launch_types<DenseBf16>(base_dtype, out_dtype, l, s);
}

}  // namespace ftmoe
