// Adapters of up to 16 ranks for few tokens: both products in one launch.
//
// Each workgroup forms h of its tile anew, from all of K, with its 16 waves,
// and then y's columns that are its own: A is read from the L2 cache by as many
// workgroups as a tile's columns make, and a launch and h's way through memory
// are saved.  B and base of the first columns are asked for before h is known.
#include "adapters_device.h"

namespace ftmoe {

namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kBatch = 4;  // units of 64 elements of K that a wave has on their way

template <typename D, typename B, typename Y>
__global__ __launch_bounds__(kThreads) void k_adapters_few(Adapters l) {
  typedef typename D::elem E;
  typedef B base8 __attribute__((ext_vector_type(8)));
  typedef base8 __attribute__((aligned(1))) base8_any;
  typedef u32x4 __attribute__((aligned(1))) any;
  constexpr int kParts = kAdapterParts<E, Y>, kFrags = (kParts + 1) / 2, kStep = 32 * kWaves;
  __shared__ float sums[kWaves][256];  // of a wave's units: rank 4 q + i of token lane % 16 at 4 lane + i
  __shared__ float total[256];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, q = lane >> 4;
  TileTokens<1> t;
  int piece = 0;
  if (!few_tile(l, blockIdx.x, l.out_each, true, t, piece)) return;
  const bool on = t.id != l.count, live = (lane & 15) < t.count;
  const float given = on && l.scale ? gload<float>(l.scale + t.id) : 1.f;
  const int wide = kStep * l.out_blocks, c0 = piece * wide;
  const int n0 = c0 + 32 * wave, n1 = min(l.out - c0, wide) + c0;

  // B's rows and base's columns as k_adapters_out takes them
  const int mine = 8 * ((lane & 15) >> 2) + (lane & 3);
  const E* weights = static_cast<const E*>(l.b) + (int64_t(t.id) * l.out + mine) * l.ld_b;
  const B* base = static_cast<const B*>(l.base) + int64_t(t.token[0]) * l.ld_base;
  Y* y = static_cast<Y*>(l.y) + int64_t(t.token[0]) * l.ld_y;
  u32x4 b[2] = {};
  base8 with = {};
  auto fetch = [&](int n) {
    if (on) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
        b[j] = row_piece<E, false>(weights + int64_t(min(n + 4 * j, l.out - 1 - mine)) * l.ld_b, q & 1, l.rank);
    }
    if (l.base) {
      const int c = n + 8 * q;
      if (c + 8 <= l.out) with = gload<base8_any>(base + c);
      else with = last_columns(base, c, l.out);
    }
  };
  if (n0 < n1) fetch(n0);

  u32x4 h[kFrags] = {};
  float scale = 0.f;
  if (on) {
    const E* x = static_cast<const E*>(l.x) + int64_t(t.token[0]) * l.ld_x;
    const E* a = static_cast<const E*>(l.a) + (int64_t(t.id) * l.rank + min(lane & 15, l.rank - 1)) * l.ld_a;
    floatx4 acc{};
    const int full = l.in / 64, units = (l.in + 63) / 64;
    for (int u0 = wave; u0 < full; u0 += kBatch * kWaves) {
      u32x4 xv[kBatch][2], av[kBatch][2];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int k = 64 * min(u0 + i * kWaves, full - 1) + 8 * q;  // (a last unit again: not added)
#pragma unroll
        for (int s = 0; s < 2; ++s) xv[i][s] = gload<any>(x + k + 32 * s);
#pragma unroll
        for (int s = 0; s < 2; ++s) av[i][s] = gload<any>(a + k + 32 * s);
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        if (u0 + i * kWaves >= full) break;
        acc = D::mfma16(av[i][0], xv[i][0], acc);
        acc = D::mfma16(av[i][1], xv[i][1], acc);
      }
    }
    if (full < units && full % kWaves == wave) {
#pragma nounroll
      for (int s = 0; s < 2; ++s) {
        const int c = 8 * full + 4 * s + q;
        acc = D::mfma16(row_piece<E, false>(a, c, l.in), row_piece<E, true>(x, c, l.in), acc);
      }
    }
    *reinterpret_cast<floatx4*>(&sums[wave][4 * lane]) = acc;
    __syncthreads();
    if (threadIdx.x < 256) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) v += sums[w][threadIdx.x];
      total[threadIdx.x] = v;
    }
    __syncthreads();
    // this lane's token, ranks 8 (q mod 2) ..; a row's last piece as row_piece takes it of B
    float v[8];
    const int c = 8 * (q & 1), from = min(c, max(l.rank - 8, 0));
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int r = from + i;
      const float s = total[64 * (r >> 2) + 4 * (lane & 15) + (r & 3)];
      v[i] = r >= c && r < l.rank ? s : 0.f;
    }
    scale = given;
    if constexpr (__is_same(E, _Float16)) scale *= to_half_range(v);
    pack_parts<E, kParts>(v, q, h);
  }

  for (int n = n0; n < n1; n += kStep) {
    float v[8] = {};
    if (l.base) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = float(with[i]);
    }
    if (on) {
      floatx4 acc[2] = {};
#pragma unroll
      for (int f = 0; f < kFrags; ++f)
#pragma unroll
        for (int j = 0; j < 2; ++j) acc[j] = D::mfma16(b[j], h[f], acc[j]);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = fmaf(acc[i >> 2][i & 3], scale, v[i]);
    }
    const int c = n + 8 * q;
    if (live && c < l.out) dense_store<Y, 8>(reinterpret_cast<uint8_t*>(y + c), 0, v, min(8, l.out - c));
    if (n + kStep < n1) fetch(n + kStep);
  }
}

template <typename D>
hipError_t launch_types(int base_dtype, int out_dtype, const Adapters& l, hipStream_t s) {
  typedef typename D::elem E;
  const dim3 grid(l.out_window.by), threads(kThreads);
  if (out_dtype == FT_DT_F32) hipLaunchKernelGGL((k_adapters_few<D, float, float>), grid, threads, 0, s, l);
  else if (base_dtype == FT_DT_F32) hipLaunchKernelGGL((k_adapters_few<D, float, E>), grid, threads, 0, s, l);
  else hipLaunchKernelGGL((k_adapters_few<D, E, E>), grid, threads, 0, s, l);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_adapters_few(int dtype, int base_dtype, int out_dtype, const Adapters& l, hipStream_t s) {
  return dtype == FT_DT_F16 ? launch_types<DenseF16>(base_dtype, out_dtype, l, s)
                            : launch_types<DenseBf16>(base_dtype, out_dtype, l, s);
}

}  // namespace ftmoe
