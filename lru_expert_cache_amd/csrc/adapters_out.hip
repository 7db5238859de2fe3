// Adapters: the second product, y = base + scale B h.
//
// Bound by reading base and writing y: 8192 tokens, N 7168, bf16: 68 us at
// rank 64, 60 at rank 16, 58 with no adapter at all (235 MB; 48 at a copy's
// rate, whose rows lie side by side); a 32-bit base 90, a 32-bit y too 124.
// 32 tokens of 32 adapters, N 6144, rank 16: 6.9 us, latency: ids, then B, base
// and h together, h's way through LDS, the products, the stores.  Ranks above
// 128: tiles of 16 tokens alone are built, 8192 tokens at rank 256 take 227 us.
// Not kept: a wave for 16 tokens and no LDS (97
// us: too little of base on its way), loads past the L2 cache (10% slower),
// three waves a SIMD by spilling (125 us).
#include "adapters_device.h"

namespace ftmoe {

namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;

// KS: steps of 32 ranks; 0: up to 16 ranks, two parts in a step
template <typename D, typename B, typename Y, int SUB, int KS>
__global__ __launch_bounds__(kThreads, SUB == 1 && KS == 0 ? 4 : 1) void k_adapters_out(Adapters l) {
  typedef typename D::elem E;
  typedef float float8 __attribute__((ext_vector_type(8)));
  typedef float8 __attribute__((aligned(4))) float8_any;
  typedef B base8 __attribute__((ext_vector_type(8)));
  constexpr bool kHalf = __is_same(E, _Float16);
  constexpr int kParts = kAdapterParts<E, Y>;
  constexpr int kSteps = KS == 0 ? 1 : KS;                          // of B's pieces
  constexpr int kFrags = KS == 0 ? (kParts + 1) / 2 : KS * kParts;  // of h's
  constexpr int kBlocks = adapter_out_blocks(sizeof(B), sizeof(Y), SUB, 32 * KS), kStep = 32 * kBlocks * kWaves;
  // sums of h: one for each group of 16 tokens and step of ranks, in kGroups shares of the parts of K
  constexpr int kGroups = SUB * kSteps >= kWaves ? 1 : kWaves / (SUB * kSteps), kSlots = SUB * kSteps * kGroups;
  // h's operands are kept in LDS where they would take many registers, made by one wave for all
  constexpr bool kShare = SUB * kFrags > 4;
  constexpr int kKept = kShare ? 1 : SUB;
  __shared__ floatx4 sums[kSlots][2][64];
  __shared__ u32x4 shared_h[kShare ? SUB * kFrags : 1][64];
  __shared__ float shared_scale[kShare ? SUB : 1][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, q = lane >> 4;
  for (uint32_t round = blockIdx.x; round < uint32_t(l.windows) * l.out_window.by; round += gridDim.x) {
    TileTokens<SUB> t;
    int piece = 0;
    if (!find_tile<SUB>(l, round, l.out_window, l.out_each, true, t, piece)) continue;
    const int wide = kStep * l.out_blocks, c0 = piece * wide;
    const int n0 = c0 + 32 * kBlocks * wave, n1 = min(l.out - c0, wide) + c0;
    const bool on = t.id != l.count;
    const float given = on && l.scale ? gload<float>(l.scale + t.id) : 1.f;

    // The parts of h, added up by the four waves together.  A lane has its
    // token's ranks 8 (q mod 2) .. for KS 0, else 32 step + 8 q ..; a row's
    // last pieces as row_piece takes them of B.
    u32x4 h[kKept][kFrags] = {};
    float scale[kKept] = {};
    auto operands = [&](int m, u32x4(&out)[kFrags], float& factor) {
      float v[kSteps * 8];
#pragma unroll
      for (int k = 0; k < kSteps; ++k) {
        const int slot = (m * kSteps + k) * kGroups;
        floatx4 lo = sums[slot][0][lane], hi = sums[slot][1][lane];
#pragma unroll
        for (int g = 1; g < kGroups; ++g) {
          lo += sums[slot + g][0][lane];
          hi += sums[slot + g][1][lane];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[8 * k + i] = lo[i];
          v[8 * k + 4 + i] = hi[i];
        }
      }
      factor = given;
      if constexpr (kHalf) factor *= to_half_range(v);
      if constexpr (KS == 0) {
        pack_parts<E, kParts>(v, q, out);
      } else {
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          u32x4 part[kParts];
          split_parts<E, kParts>(v + 8 * k, part);
#pragma unroll
          for (int p = 0; p < kParts; ++p) out[k * kParts + p] = part[p];
        }
      }
    };
    auto join = [&]() {
      __syncthreads();  // the last tile's are done with
#pragma unroll
      for (int i = 0; i < kSlots / kWaves; ++i) {
        const int slot = wave + kWaves * i, m = slot / kGroups / kSteps, k = slot / kGroups % kSteps;
        const int c = KS == 0 ? (q & 1) : 4 * k + q;
        const float* row = l.h + int64_t(t.token[0]) * l.ld_h;
#pragma unroll
        for (int n = 1; n < SUB; ++n) row = m == n ? l.h + int64_t(t.token[n]) * l.ld_h : row;
        const int64_t part = int64_t(l.tokens) * l.ld_h;
        const int from = min(8 * c, max(l.rank - 8, 0));
        float8 sum{};
        if (8 * c < l.rank) {
          if (l.rank >= 8) {
#pragma unroll 4
            for (int p = slot % kGroups; p < l.parts; p += kGroups) sum += gload<float8_any>(row + p * part + from);
#pragma unroll
            for (int e = 0; e < 8; ++e) sum[e] = from + e >= 8 * c ? sum[e] : 0.f;
          } else {
            for (int p = slot % kGroups; p < l.parts; p += kGroups) {
#pragma unroll
              for (int e = 0; e < 8; ++e)
                if (e < l.rank) sum[e] += gload<float>(row + p * part + e);
            }
          }
        }
        sums[slot][0][lane] = __builtin_shufflevector(sum, sum, 0, 1, 2, 3);
        sums[slot][1][lane] = __builtin_shufflevector(sum, sum, 4, 5, 6, 7);
      }
      __syncthreads();
      if constexpr (kShare) {
        for (int m = wave; m < SUB; m += kWaves) {
          u32x4 made[kFrags];
          float factor;
          operands(m, made, factor);
#pragma unroll
          for (int f = 0; f < kFrags; ++f) shared_h[m * kFrags + f][lane] = made[f];
          shared_scale[m][lane] = factor;
        }
        __syncthreads();
      } else {
#pragma unroll
        for (int m = 0; m < SUB; ++m) operands(m, h[m], scale[m]);
      }
    };

    // A block's 32 columns: two instructions, whose rows 4 a + i are columns 8 a + 4 j + i: lane (q, token) gets
    // columns 8 q .. 8 q + 7.  A wave takes as many blocks at once as fill a cache line of base and y.
    u32x4 b[kBlocks][2][kSteps] = {};
    base8 with[SUB][kBlocks] = {};
    const int mine = 8 * ((lane & 15) >> 2) + (lane & 3);
    auto fetch = [&](int n) {
      if (on) {
#pragma unroll
        for (int w = 0; w < kBlocks; ++w) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int64_t at = int64_t(t.id) * l.out + min(n + 32 * w + mine + 4 * j, l.out - 1);
            const E* row = static_cast<const E*>(l.b) + at * l.ld_b;
#pragma unroll
            for (int k = 0; k < kSteps; ++k) b[w][j][k] = row_piece<E, false>(row, KS == 0 ? (q & 1) : 4 * k + q, l.rank);
          }
        }
      }
      if (l.base) {
#pragma unroll
        for (int m = 0; m < SUB; ++m) {
          const B* row = static_cast<const B*>(l.base) + int64_t(t.token[m]) * l.ld_base;
          typedef base8 __attribute__((aligned(1))) any;
#pragma unroll
          for (int w = 0; w < kBlocks; ++w) {
            const int c = n + 32 * w + 8 * q;
            if (c + 8 <= l.out) with[m][w] = gload<any>(row + c);
            else with[m][w] = last_columns(row, c, l.out);
          }
        }
      }
    };
    for (int n = n0 - kStep; n < n1; n += kStep) {  // each step's loads are a turn ahead of its products
      u32x4 bn[kBlocks][2][kSteps];
      base8 wn[SUB][kBlocks];
#pragma unroll
      for (int w = 0; w < kBlocks; ++w) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int k = 0; k < kSteps; ++k) bn[w][j][k] = b[w][j][k];
#pragma unroll
        for (int m = 0; m < SUB; ++m) wn[m][w] = with[m][w];
      }
      if (n + kStep < n1) fetch(n + kStep);
      if (n < n0) {  // the first turn, of every wave
        if (on) join();
        continue;
      }
#pragma unroll
      for (int m = 0; m < SUB; ++m) {
        u32x4 hm[kFrags];
        float factor = 0.f;
        if (on) {
#pragma unroll
          for (int f = 0; f < kFrags; ++f) hm[f] = kShare ? shared_h[m * kFrags + f][lane] : h[kShare ? 0 : m][f];
          factor = kShare ? shared_scale[m][lane] : scale[kShare ? 0 : m];
        }
#pragma unroll
        for (int w = 0; w < kBlocks; ++w) {
          const int c = n + 32 * w + 8 * q;
          float v[8] = {};
          if (on) {
            floatx4 acc[2] = {};
#pragma unroll
            for (int f = 0; f < kFrags; ++f)
#pragma unroll
              for (int j = 0; j < 2; ++j) acc[j] = D::mfma16(bn[w][j][KS == 0 ? 0 : f / kParts], hm[f], acc[j]);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = acc[i >> 2][i & 3] * factor;
          }
          if (l.base) {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] += float(wn[m][w][i]);
          }
          if (16 * m + (lane & 15) < t.count && c < l.out)
            dense_store<Y, 8>(static_cast<uint8_t*>(l.y), int64_t(t.token[m]) * l.ld_y + c, v, min(8, l.out - c));
        }
      }
    }
  }
}

template <typename D, typename B, typename Y, int SUB, int KS>
hipError_t launch(const Adapters& l, hipStream_t s) {
  hipLaunchKernelGGL((k_adapters_out<D, B, Y, SUB, KS>), dim3(adapter_grid(adapter_rounds(l, l.out_window))), dim3(kThreads), 0, s, l);
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
    if (ks == 2) return launch<D, B, Y, 2, 2>(l, s);
    return launch<D, B, Y, 2, 4>(l, s);
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
