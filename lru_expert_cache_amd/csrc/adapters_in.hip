// Adapters: tiles of tokens, and the first product, h = A x.
//
// The product is bound by reading x: a few ranks make two operations of each
// byte.  8192 tokens, K 7168, a fifth of them without an adapter, bf16: 36 us
// at rank 64 (94 MB of x and as much of A from the L2 cache), 29 at rank 16,
// against 19 for x at a copy's rate; 32 tokens of 32 adapters, K 6144, rank
// 16: 4.0 us (6 MB of A), half of it latency.  Grouping takes 4.4 us for 1531
// tokens and 8 for 8192, in one workgroup a window.
#include "adapters_device.h"

namespace ftmoe {

namespace {

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int kPlanThreads = 1024, kEach = kAdapterWindow / kPlanThreads;

// The tiles of a window: tokens are counted by adapter (those without one last),
// and placed at their adapter's offset.  Which place within it a token gets
// depends on the order of the atomics; its result does not.
__global__ __launch_bounds__(kPlanThreads) void k_adapters_plan(Adapters l) {
  extern __shared__ int lds[];
  __shared__ uint32_t sums[kPlanThreads / 64];
  int* hist = lds;                                               // [count + 1]
  uint32_t* before = reinterpret_cast<uint32_t*>(lds) + l.count + 1;  // [count + 1]: tokens, and tiles above
  const int tid = threadIdx.x, lane = tid & 63, groups = l.count + 1;
  const int size = 16 * l.sub, shift = l.sub == 1 ? 4 : l.sub == 2 ? 5 : 6;  // tokens of a tile, a power of two
  const int64_t t0 = int64_t(blockIdx.x) * kAdapterWindow;
  const int tokens = int(min(int64_t(kAdapterWindow), l.tokens - t0));
  for (int g = tid; g < groups; g += kPlanThreads) hist[g] = 0;
  // eight tokens a thread, in two loads where they are all there
  int group[kEach], place[kEach];
  {
    static_assert(kEach == 8, "two loads");
    typedef int intx4_any __attribute__((ext_vector_type(4), aligned(4)));
    const int32_t* ids = l.ids + t0 + kEach * tid;
    if (kEach * tid + kEach <= tokens) {
      const intx4_any a = gload<intx4_any>(ids), b = gload<intx4_any>(ids + 4);
#pragma unroll
      for (int i = 0; i < kEach; ++i) group[i] = i < 4 ? a[i & 3] : b[i & 3];
    } else {
#pragma unroll
      for (int i = 0; i < kEach; ++i) group[i] = kEach * tid + i < tokens ? gload<int32_t>(ids + i) : -1;
    }
#pragma unroll
    for (int i = 0; i < kEach; ++i) {
      const bool bare = uint32_t(group[i]) >= uint32_t(l.count);
      group[i] = kEach * tid + i >= tokens || (bare && l.in_place) ? -1 : bare ? l.count : group[i];
    }
  }
  __syncthreads();
  // One addition for each run of the same adapter: lanes whose tokens are all
  // of one, and of the same as the lane's before, leave it to the first of
  // them (an addition for each lane of a long prompt took 3 us more).
  bool whole = group[0] >= 0;
#pragma unroll
  for (int i = 1; i < kEach; ++i) whole = whole && group[i] == group[0];
  const int before_whole = __shfl_up(int(whole), 1), before_group = __shfl_up(group[0], 1);  // by every lane
  const bool follows = whole && lane > 0 && before_whole && before_group == group[0];
  const uint64_t heads = ~__ballot(follows);
  const int head = 63 - __builtin_clzll(heads & (~uint64_t(0) >> (63 - lane)));
  const uint64_t later = heads >> lane >> 1;  // this lane's run ends before the next head
  const int lanes = later ? __builtin_ctzll(later) + 1 : 64 - lane;
  int base = 0;
  if (whole && !follows) base = atomicAdd(&hist[group[0]], kEach * lanes);
  base = __shfl(base, head) + kEach * (lane - head);
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    place[i] = base + i;
    if (whole) continue;
    if (i > 0 && group[i] == group[i - 1]) {
      place[i] = place[i - 1] + 1;
    } else if (group[i] >= 0) {
      int run = 1;
      bool on = true;
#pragma unroll
      for (int j = i + 1; j < kEach; ++j) {
        on = on && group[j] == group[i];
        run += on;
      }
      place[i] = atomicAdd(&hist[group[i]], run);
    }
  }
  __syncthreads();
  // a window's tokens and tiles fit 16 bits each
  const int each = (groups + kPlanThreads - 1) / kPlanThreads;
  uint32_t own = 0;
  for (int j = 0; j < each; ++j) {
    const int g = tid * each + j, c = g < groups ? hist[g] : 0;
    own += uint32_t(c) + (uint32_t((c + size - 1) >> shift) << 16);
  }
  uint32_t sum = own;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const uint32_t v = __shfl_up(sum, o);
    sum += lane >= o ? v : 0;
  }
  if (lane == 63) sums[tid >> 6] = sum;
  __syncthreads();
  uint32_t at = sum - own;
  for (int i = 0; i < tid >> 6; ++i) at += sums[i];
  if (tid == kPlanThreads - 1) {
    const int all = int((at + own) >> 16);
    l.tile_count[2 * blockIdx.x] = all;
    l.tile_count[2 * blockIdx.x + 1] = all - ((hist[l.count] + size - 1) >> shift);
  }
  for (int j = 0; j < each; ++j) {
    const int g = tid * each + j;
    if (g >= groups) break;
    before[g] = at;
    const int c = hist[g];
    at += uint32_t(c) + (uint32_t((c + size - 1) >> shift) << 16);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int g = group[i];
    if (g < 0) continue;
    const uint32_t b = before[g];
    const int first = int(t0) + int(b & 0xFFFF) + place[i];
    l.order[first] = int(t0) + kEach * tid + i;
    if ((place[i] & (size - 1)) == 0)
      l.tiles[int64_t(blockIdx.x) * l.tile_cap + (b >> 16) + (place[i] >> shift)] = {g, first, min(size, hist[g] - place[i]), 0};
  }
}

// A workgroup takes a tile of tokens, up to 64 rows of its adapter's A and a
// part of K, which its four waves share; their sums meet in LDS.  A matrix
// instruction takes 16 rows of A and 16 tokens, 16 bytes of each row a lane:
// half of a row's cache line, so both halves are asked for one after the other
// (half of every 16 rows first, then the others: 42 us for the 36 above, with
// half as many requests again to the L2 cache).
template <typename D, int SUB, int ROWS>
__global__ __launch_bounds__(kThreads) void k_adapters_in(Adapters l) {
  typedef typename D::elem E;
  __shared__ floatx4 lds[kWaves][SUB * ROWS][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, q = lane >> 4;
  for (uint32_t round = blockIdx.x; round < uint32_t(l.windows) * l.in_window.by; round += gridDim.x) {
    TileTokens<SUB> t;
    int piece = 0;
    if (!find_tile<SUB>(l, round, l.in_window, l.in_each, false, t, piece)) continue;
    const int block = int(l.by_parts(uint32_t(piece))), part = piece - block * l.parts;
    const E* x[SUB];
    const E* a[ROWS];
#pragma unroll
    for (int m = 0; m < SUB; ++m) x[m] = static_cast<const E*>(l.x) + int64_t(t.token[m]) * l.ld_x;
#pragma unroll
    for (int j = 0; j < ROWS; ++j) {
      const int r = min(16 * (block * ROWS + j) + (lane & 15), l.rank - 1);
      a[j] = static_cast<const E*>(l.a) + (int64_t(t.id) * l.rank + r) * l.ld_a;
    }
    // K in units of 64 elements: two instructions, 128 bytes of a row
    const uint32_t units = uint32_t(l.in + 63) / 64;  // times a part's number: below 2^31
    const uint32_t p0 = l.by_parts(units * part), p1 = l.by_parts(units * (part + 1));
    // the waves take units in turn: 512 bytes of each row are asked for at about the same time
    const int u0 = int(p0) + wave, u1 = int(min(p1, uint32_t(l.in) / 64));
    const bool tail = p1 == units && l.in % 64 != 0 && (int(units) - 1 - u0) % kWaves == 0 && u0 < int(units);
    floatx4 acc[SUB][ROWS] = {};
    auto step = [&](const u32x4(&xv)[SUB], const u32x4(&av)[ROWS]) {
#pragma unroll
      for (int m = 0; m < SUB; ++m)
#pragma unroll
        for (int j = 0; j < ROWS; ++j) acc[m][j] = D::mfma16(av[j], xv[m], acc[m][j]);
    };
    typedef u32x4 __attribute__((aligned(1))) any;
    u32x4 xv[2][SUB] = {}, av[2][ROWS] = {};
    auto fetch = [&](int u) {
      // both halves of a line next to each other
      const int k = 64 * u + 8 * q;
#pragma unroll
      for (int m = 0; m < SUB; ++m)
#pragma unroll
        for (int h = 0; h < 2; ++h) xv[h][m] = gload<any>(x[m] + k + 32 * h);
#pragma unroll
      for (int j = 0; j < ROWS; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h) av[h][j] = gload<any>(a[j] + k + 32 * h);
    };
    if (u0 < u1) fetch(u0);
    for (int u = u0; u < u1; u += kWaves) {
      u32x4 xn[2][SUB], an[2][ROWS];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int m = 0; m < SUB; ++m) xn[h][m] = xv[h][m];
#pragma unroll
        for (int j = 0; j < ROWS; ++j) an[h][j] = av[h][j];
      }
      if (u + kWaves < u1) fetch(u + kWaves);
      step(xn[0], an[0]);
      step(xn[1], an[1]);
    }
    if (tail) {
#pragma nounroll
      for (int h = 0; h < 2; ++h) {
        const int c = 8 * (int(units) - 1) + 4 * h + q;
#pragma unroll
        for (int m = 0; m < SUB; ++m) xv[0][m] = row_piece<E, true>(x[m], c, l.in);
#pragma unroll
        for (int j = 0; j < ROWS; ++j) av[0][j] = row_piece<E, false>(a[j], c, l.in);
        step(xv[0], av[0]);
      }
    }
    __syncthreads();  // the last tile's sums have been read
#pragma unroll
    for (int m = 0; m < SUB; ++m)
#pragma unroll
      for (int j = 0; j < ROWS; ++j) lds[wave][m * ROWS + j][lane] = acc[m][j];
    __syncthreads();
#pragma unroll
    for (int m = 0; m < SUB; ++m) {
#pragma unroll
      for (int j = 0; j < ROWS; ++j) {
        if ((m * ROWS + j) % kWaves != wave) continue;
        floatx4 v = lds[0][m * ROWS + j][lane];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) v += lds[w][m * ROWS + j][lane];
        const int r = 16 * (block * ROWS + j) + 4 * q;
        float* h = l.h + (int64_t(part) * l.tokens + t.token[m]) * l.ld_h + r;
        // h's rows hold whole groups of four
        if (16 * m + (lane & 15) < t.count && r < l.ld_h) gstore<floatx4>(h, v);
      }
    }
  }
}

template <typename D, int SUB, int ROWS>
hipError_t launch(const Adapters& l, hipStream_t s) {
  hipLaunchKernelGGL((k_adapters_in<D, SUB, ROWS>), dim3(adapter_grid(adapter_rounds(l, l.in_window))), dim3(kThreads), 0, s, l);
  return hipGetLastError();
}
template <typename D, int SUB>
hipError_t launch_rank(const Adapters& l, hipStream_t s) {
  if (l.rank <= 16) return launch<D, SUB, 1>(l, s);
  if (l.rank <= 32) return launch<D, SUB, 2>(l, s);
  return launch<D, SUB, 4>(l, s);
}
template <typename D>
hipError_t launch_sub(const Adapters& l, hipStream_t s) {
  if (l.sub == 1) return launch_rank<D, 1>(l, s);
  if (l.sub == 2) return launch_rank<D, 2>(l, s);
  return launch_rank<D, 4>(l, s);
}

}  // namespace

hipError_t launch_adapters_plan(const Adapters& l, hipStream_t s) {
  hipLaunchKernelGGL(k_adapters_plan, dim3(uint32_t(l.windows)), dim3(kPlanThreads), size_t(l.count + 1) * 8, s, l);
  return hipGetLastError();
}
hipError_t launch_adapters_in(int dtype, const Adapters& l, hipStream_t s) {
  return dtype == FT_DT_F16 ? launch_sub<DenseF16>(l, s) : launch_sub<DenseBf16>(l, s);
}

}  // namespace ftmoe
