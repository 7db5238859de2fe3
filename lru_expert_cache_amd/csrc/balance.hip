// A router's balance: choice, weights, counts and loss of a batch of tokens, and the gradient of the logits.
//
// A wave takes a token at a time; lane l holds experts l, l + 64, ..., sorted.
// The k largest are found in k rounds: the maximum over the lanes' first ones
// (as integers of the logits' order, reduced with DPP: no LDS round trips),
// the lane that has it from a ballot, and that lane moves up its next.
// The sums over the tokens are kept by each lane for its experts, added up
// within the workgroup, and over the workgroups, in order, by a second kernel
// (up to 32 tokens are one workgroup's, which writes counts and loss itself).
//
// 32768 tokens, 256 experts, top 8: 25.9 us (floor 7: the logits once), bound by
// the vector units (397 instructions a token; 41 us when each round looked
// through all of a lane's logits); the join 6.7; the gradient 17.0 (floor 14),
// bound by HBM and the vector units (208).  509 tokens, 128 experts: 4.3, 5.6
// and 3.7 us, all latency.
#include <type_traits>

#include "balance.h"

namespace ftmoe {

namespace {

// One workgroup, and no second launch, up to this many tokens: choice, loss and gradient of 16 / 32 / 64 tokens, 128
// experts, in a graph 8.3 / 10.8 / 15.0 us, with a second launch 11.5 / 11.5 / 11.7 (with shorter exponentials).
constexpr int kOne = 32;
// waves of a workgroup: few tokens are spread over more CUs (509 tokens, 128 experts: 4.4 us against 5.0 with 16
// waves), many leave fewer parts to add up
constexpr int balance_waves(int32_t tokens) { return tokens <= 4 || (tokens > kOne && tokens <= 2048) ? 4 : 16; }
constexpr int kBackWaves = 4;
constexpr float kInf = __builtin_huge_valf();
constexpr uint32_t kNever = 0;  // below every logit that can be chosen

// lanes' partners within a row of 16, then lane 15 of a row to the next, lane 31 to the upper half: lane 63 has all
template <int CTRL, int ROWS = 0xF>
__device__ __attribute__((always_inline)) inline uint32_t dpp(uint32_t v) {
  return uint32_t(__builtin_amdgcn_update_dpp(0, int(v), CTRL, ROWS, 0xF, false));
}
__device__ __attribute__((always_inline)) inline uint32_t wave_top(uint32_t v) {
  v = max(v, dpp<0xB1>(v));
  v = max(v, dpp<0x4E>(v));
  v = max(v, dpp<0x141>(v));
  v = max(v, dpp<0x140>(v));
  v = max(v, dpp<0x142, 0xA>(v));
  v = max(v, dpp<0x143, 0xC>(v));
  return uint32_t(__builtin_amdgcn_readlane(int(v), 63));
}
__device__ __attribute__((always_inline)) inline float wave_sum(float x) {
  auto all = [](float v, auto ctrl) {
    return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), decltype(ctrl)::value, 0xF, 0xF, true));
  };
  x += all(x, std::integral_constant<int, 0xB1>{});
  x += all(x, std::integral_constant<int, 0x4E>{});
  x += all(x, std::integral_constant<int, 0x141>{});
  x += all(x, std::integral_constant<int, 0x140>{});
  x += __uint_as_float(dpp<0x142, 0xA>(__float_as_uint(x)));
  x += __uint_as_float(dpp<0x143, 0xC>(__float_as_uint(x)));
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(x), 63));
}

// Logits as integers of their order (-0 as 0); -inf and NaN, which are never chosen, below all.
__device__ __attribute__((always_inline)) inline uint32_t order_of(float z) {
  const int b = __float_as_int(z + 0.f);
  const uint32_t k = uint32_t(b) ^ (uint32_t(b >> 31) | 0x80000000u);
  return z > -kInf ? k : kNever;
}
__device__ __attribute__((always_inline)) inline float logit_of(uint32_t k) {
  return __uint_as_float(k ^ (uint32_t(int(~k) >> 31) | 0x80000000u));
}

// e^d, d <= 0, to within two units at any distance, subnormal results too: d = n ln 2 + r, ln 2 in two parts (a single
// product d log2 e rounds by up to |d| / 2 units, and the hardware's exp2 leaves 0 below 2^-126).  Below -104 it is 0.
// All of a router's step over 32768 tokens and 256 experts: 47.4 us; by that product and the bare reciprocal 43.7.
__device__ __attribute__((always_inline)) inline float exp_of(float d) {
  const float c = d < -104.f ? -104.f : d;  // NaN stays
  const float n = rintf(c * 1.4426950408889634f);
  const float r = fmaf(-n, -1.904654323148236e-09f, fmaf(-n, 0.693147182464599609375f, c));
  return ldexpf(__builtin_amdgcn_exp2f(r * 1.4426950408889634f), int(n));
}

// Quotients by v, of 1 to 512: by the hardware's reciprocal, which is off by a unit, and then by what is left over.
struct Over {
  float v, r;
  __device__ __attribute__((always_inline)) inline explicit Over(float v_) : v(v_) {
    const float near = __builtin_amdgcn_rcpf(v);
    r = fmaf(fmaf(-v, near, 1.f), near, near);
  }
  __device__ __attribute__((always_inline)) inline float operator()(float e) const {
    const float q = e * r;
    return fmaf(fmaf(-v, q, e), r, q);
  }
};

// A token's logits, J for each lane; -inf beyond the last.
template <typename X, int J>
struct Logits {
  float z[J];
  __device__ __attribute__((always_inline)) inline void load(const X* row, int experts, int lane) {
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int e = lane + 64 * j;
      const float v = float(gload<X>(row + min(e, experts - 1)));
      z[j] = e < experts ? v : -kInf;
    }
  }
  // the largest as its integer; kNever where none can be chosen
  __device__ __attribute__((always_inline)) inline uint32_t top(uint32_t (&key)[J]) const {
    uint32_t best = kNever;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      key[j] = order_of(z[j]);
      best = max(best, key[j]);
    }
    return wave_top(best);
  }
  // whether some logit is not -inf
  __device__ __attribute__((always_inline)) inline bool some(uint32_t top) const {
    if (top != kNever) return true;
    bool nan = false;
#pragma unroll
    for (int j = 0; j < J; ++j) nan = nan || z[j] != z[j];
    return __any(nan);
  }
  // softmax, the largest logit known; 0 beyond the last expert
  __device__ __attribute__((always_inline)) inline void softmax(float (&p)[J], float top, int experts, int lane) const {
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const float e = exp_of(z[j] - top);
      p[j] = lane + 64 * j < experts ? e : 0.f;
      sum += p[j];
    }
    const Over over(wave_sum(sum));
#pragma unroll
    for (int j = 0; j < J; ++j) p[j] = over(p[j]);
  }
};

// from the tokens counted and the sum of c_e sum_t p[t][e]
__device__ inline float balance_loss(const BalanceForward& a, int v, double sum) {
  const double n = double(v);
  return v ? float(double(a.weight) * a.experts / (a.top_k * n * n) * sum) : 0.f;
}

template <typename X, int J, int kWaves>
__global__ __launch_bounds__(64 * kWaves) void k_balance(BalanceForward a) {
  __shared__ float lds_p[kWaves][64 * J];
  __shared__ int lds_c[64 * J];
  __shared__ int lds_v;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);  // addresses of rows: scalar
  for (int e = threadIdx.x; e < 64 * J; e += 64 * kWaves) lds_c[e] = 0;
  if (threadIdx.x == 0) {
    lds_v = 0;
    if (blockIdx.x == 0) *a.arrived = 0;  // of the next kernel's workgroups
  }
  __syncthreads();
  float sums[J] = {};
  int counted = 0;
  const int64_t step = int64_t(a.groups) * kWaves;
  Logits<X, J> next;
  bool next_on = true;
  int64_t t = int64_t(blockIdx.x) * kWaves + wave;
  const X* row = static_cast<const X*>(a.logits) + t * a.ld;
  int32_t* sel = a.sel + t * a.top_k;
  float* w = a.w + t * a.top_k;
  auto fetch = [&](int64_t t) {
    next.load(row, a.experts, lane);
    next_on = !a.valid || gload<uint8_t>(a.valid + t);
    row += step * a.ld;
  };
  if (t < a.tokens) fetch(t);
  for (; t < a.tokens; t += step) {
    const Logits<X, J> l = next;
    const bool valid = next_on;
    if (t + step < a.tokens) fetch(t + step);
    uint32_t key[J];
    const uint32_t first = l.top(key);
    int mine = -1;  // lane i: the choice of rank i, and its logit
    uint32_t mine_key = kNever;
    if (valid && l.some(first)) {
      ++counted;
      float p[J];
      l.softmax(p, logit_of(first), a.experts, lane);
#pragma unroll
      for (int j = 0; j < J; ++j) sums[j] += p[j];
      // larger first, the lower expert first on ties (neighbours only are exchanged)
      int expert[J];
#pragma unroll
      for (int j = 0; j < J; ++j) expert[j] = lane + 64 * j;
#pragma unroll
      for (int r = 0; r < J; ++r) {
#pragma unroll
        for (int j = r & 1; j + 1 < J; j += 2) {
          const bool swap = key[j + 1] > key[j];
          const uint32_t hi = max(key[j], key[j + 1]), lo = min(key[j], key[j + 1]);
          key[j] = hi;
          key[j + 1] = lo;
          const int x = expert[j], y = expert[j + 1];
          expert[j] = swap ? y : x;
          expert[j + 1] = swap ? x : y;
        }
      }
      uint32_t best = first;
      for (int i = 0; i < a.top_k && best != kNever; ++i) {
        uint64_t same = __ballot(key[0] == best);
        int src = __builtin_ctzll(same);
        int at = __builtin_amdgcn_readlane(expert[0], src);
        for (same &= same - 1; same; same &= same - 1) {  // other lanes have that logit too
          const int s = __builtin_ctzll(same), e = __builtin_amdgcn_readlane(expert[0], s);
          if (e < at) {
            at = e;
            src = s;
          }
        }
        mine = lane == i ? at : mine;
        mine_key = lane == i ? best : mine_key;
        if (lane == src) {
#pragma unroll
          for (int j = 0; j + 1 < J; ++j) {
            key[j] = key[j + 1];
            expert[j] = expert[j + 1];
          }
          key[J - 1] = kNever;
        }
        best = wave_top(key[0]);
      }
      if (mine >= 0) atomicAdd(&lds_c[mine], 1);
    }
    const float ex = mine >= 0 ? exp_of(logit_of(mine_key) - logit_of(first)) : 0.f;
    const Over over(wave_sum(ex));
    if (lane < a.top_k) {
      sel[lane] = mine;
      w[lane] = mine >= 0 ? over(ex) : 0.f;
    }
    sel += step * a.top_k;
    w += step * a.top_k;
  }
#pragma unroll
  for (int j = 0; j < J; ++j) lds_p[wave][lane + 64 * j] = sums[j];
  if (lane == 0) atomicAdd(&lds_v, counted);
  __syncthreads();
  if (a.groups == 1) {
    // all there is: each expert's share of the loss
    double share = 0.0;
    for (int e = threadIdx.x; e < a.experts; e += 64 * kWaves) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < kWaves; ++i) s += lds_p[i][e];
      a.counts[e] = lds_c[e];
      share += double(s) * lds_c[e];
    }
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) share += __shfl_xor(share, o);
    __shared__ double lds_s[kWaves];
    if (lane == 0) lds_s[wave] = share;
    __syncthreads();
    if (threadIdx.x == 0) {
      double sum = 0.0;
#pragma unroll
      for (int i = 0; i < kWaves; ++i) sum += lds_s[i];
      a.counts[a.experts] = lds_v;
      a.loss[0] = balance_loss(a, lds_v, sum);
    }
    return;
  }
  for (int e = threadIdx.x; e < 64 * J; e += 64 * kWaves) {
    float s = 0.f;
    for (int i = 0; i < kWaves; ++i) s += lds_p[i][e];
    a.part_p[int64_t(blockIdx.x) * a.ld_part + e] = s;
    a.part_c[int64_t(blockIdx.x) * a.ld_part + e] = lds_c[e];
  }
  if (threadIdx.x == 0) a.part_v[blockIdx.x] = lds_v;
}

// Sixteen experts a workgroup: four lanes have four each, 64 groups of lanes
// every 64th part.  The workgroup that arrives last adds up the loss: the
// others' shares of it are written past the XCD's own cache, and the counter
// is touched after them.
constexpr int kJoin = 512;
__global__ __launch_bounds__(kJoin) void k_balance_join(BalanceForward a) {
  typedef float floatx4 __attribute__((ext_vector_type(4)));
  typedef int intx4 __attribute__((ext_vector_type(4)));
  __shared__ double lds_p[kJoin / 64][16];
  __shared__ int lds_c[kJoin / 64][16];
  __shared__ int last;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, col = 4 * (tid & 3);
  const int e0 = 16 * int(blockIdx.x);
  double p[4] = {};
  int c[4] = {}, v = 0;
  if (wave == 0)
    for (int g = lane; g < a.groups; g += 64) v += a.part_v[g];
#pragma unroll 4
  for (int g = tid >> 2; g < a.groups; g += kJoin / 4) {
    const floatx4 pv = gload<floatx4>(a.part_p + int64_t(g) * a.ld_part + e0 + col);
    const intx4 cv = gload<intx4>(a.part_c + int64_t(g) * a.ld_part + e0 + col);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      p[i] += double(pv[i]);
      c[i] += cv[i];
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int o = 4; o < 64; o <<= 1) {
      p[i] += __shfl_xor(p[i], o);
      c[i] += __shfl_xor(c[i], o);
    }
    if (lane < 4) {
      lds_p[wave][col + i] = p[i];
      lds_c[wave][col + i] = c[i];
    }
  }
  __syncthreads();
  if (tid < 16) {
    double ps = 0.0;
    int cs = 0;
    for (int w = 0; w < kJoin / 64; ++w) {
      ps += lds_p[w][tid];
      cs += lds_c[w][tid];
    }
    if (e0 + tid < a.experts) a.counts[e0 + tid] = cs;
    double share = ps * cs;
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) share += __shfl_xor(share, o);
    if (tid == 0) {
      __hip_atomic_store(a.share + blockIdx.x, share, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      last = __hip_atomic_fetch_add(a.arrived, 1, __ATOMIC_ACQ_REL, __HIP_MEMORY_SCOPE_AGENT) == int(gridDim.x) - 1;
    }
  }
  __syncthreads();
  if (!last || wave != 0) return;
  double sum = lane < int(gridDim.x) ? __hip_atomic_load(a.share + lane, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) : 0.0;
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) {
    v += __shfl_xor(v, o);
    sum += __shfl_xor(sum, o);
  }
  if (lane == 0) {
    a.counts[a.experts] = v;
    a.loss[0] = balance_loss(a, v, sum);
  }
}

template <typename X, int J>
__global__ __launch_bounds__(64 * kBackWaves) void k_balance_backward(BalanceBackward a) {
  __shared__ float lds[kBackWaves][64 * J];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  float c[J];
  {
    const double v = double(a.counts[a.experts]);
    const double k = v > 0 ? double(a.weight) * a.experts / (a.top_k * v * v) : 0.0;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int e = lane + 64 * j;
      c[j] = e < a.experts ? float(k * a.counts[e]) : 0.f;
      lds[wave][e] = 0.f;
    }
  }
  const float dloss = a.dloss ? a.dloss[0] : 1.f;
  const int64_t step = int64_t(gridDim.x) * kBackWaves;
  Logits<X, J> next;
  bool next_on = true;
  int next_sel = -1;
  float next_w = 0.f, next_dw = 0.f;
  auto fetch = [&](int64_t t) {
    next.load(static_cast<const X*>(a.logits) + t * a.ld, a.experts, lane);
    next_on = !a.valid || gload<uint8_t>(a.valid + t);
    if (a.dw && lane < a.top_k) {
      next_sel = gload<int>(a.sel + t * a.top_k + lane);
      next_w = gload<float>(a.w + t * a.top_k + lane);
      next_dw = gload<float>(a.dw + t * a.top_k + lane);
    }
  };
  int64_t t = int64_t(blockIdx.x) * kBackWaves + wave;
  if (t < a.tokens) fetch(t);
  for (; t < a.tokens; t += step) {
    const Logits<X, J> l = next;
    const bool valid = next_on;
    const int i = next_sel;
    const bool chosen = uint32_t(i) < uint32_t(a.experts);
    const float w = chosen ? next_w : 0.f, dw = chosen ? next_dw : 0.f;
    if (t + step < a.tokens) fetch(t + step);
    X* dz = static_cast<X*>(a.dlogits) + t * a.ld;
    float d[J] = {};
    uint32_t key[J];
    const uint32_t top = l.top(key);
    if (valid && l.some(top)) {
      float p[J], sum = 0.f;
      l.softmax(p, logit_of(top), a.experts, lane);
#pragma unroll
      for (int j = 0; j < J; ++j) sum = fmaf(p[j], c[j], sum);
      sum = wave_sum(sum);
#pragma unroll
      for (int j = 0; j < J; ++j) d[j] = dloss * p[j] * (c[j] - sum);
      if (a.dw) {
        const float mean = wave_sum(w * dw);
        if (chosen) atomicAdd(&lds[wave][i], w * (dw - mean));  // the same expert twice counts twice
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int j = 0; j < J; ++j) d[j] += lds[wave][lane + 64 * j];
        __builtin_amdgcn_wave_barrier();
        if (chosen) lds[wave][i] = 0.f;
        __builtin_amdgcn_wave_barrier();
      }
    }
#pragma unroll
    for (int j = 0; j < J; ++j)
      if (lane + 64 * j < a.experts) gstore<X>(dz + lane + 64 * j, X(d[j]));
  }
}

template <typename X, int J>
hipError_t launch(const BalanceForward& a, hipStream_t s) {
  if (a.ld_part != 64 * J) return hipErrorInvalidValue;
  if (balance_waves(a.tokens) == 4)
    hipLaunchKernelGGL((k_balance<X, J, 4>), dim3(uint32_t(a.groups)), dim3(64 * 4), 0, s, a);
  else
    hipLaunchKernelGGL((k_balance<X, J, 16>), dim3(uint32_t(a.groups)), dim3(64 * 16), 0, s, a);
  if (a.groups == 1) return hipGetLastError();
  hipLaunchKernelGGL(k_balance_join, dim3(uint32_t((a.experts + 15) / 16)), dim3(kJoin), 0, s, a);
  return hipGetLastError();
}
template <typename X, int J>
hipError_t launch(const BalanceBackward& a, hipStream_t s) {
  const int32_t groups = (a.tokens + kBackWaves - 1) / kBackWaves;
  hipLaunchKernelGGL((k_balance_backward<X, J>), dim3(uint32_t(groups < 2048 ? groups : 2048)), dim3(64 * kBackWaves), 0, s, a);
  return hipGetLastError();
}
template <typename X, typename A>
hipError_t launch_width(const A& a, hipStream_t s) {
  if (a.experts <= 64) return launch<X, 1>(a, s);
  if (a.experts <= 128) return launch<X, 2>(a, s);
  if (a.experts <= 256) return launch<X, 4>(a, s);
  return launch<X, 8>(a, s);
}
template <typename A>
hipError_t launch_type(int dtype, const A& a, hipStream_t s) {
  if (dtype == FT_DT_F32) return launch_width<float>(a, s);
  if (dtype == FT_DT_F16) return launch_width<_Float16>(a, s);
  return launch_width<__bf16>(a, s);
}

}  // namespace

int balance_groups(int32_t tokens) {
  if (tokens <= kOne) return 1;
  const int32_t waves = balance_waves(tokens), g = (tokens + waves - 1) / waves;
  return g < 512 ? g : 512;
}

hipError_t launch_balance(int dtype, const BalanceForward& a, hipStream_t s) { return launch_type(dtype, a, s); }
hipError_t launch_balance_backward(int dtype, const BalanceBackward& a, hipStream_t s) {
  return launch_type(dtype, a, s);
}

}  // namespace ftmoe
