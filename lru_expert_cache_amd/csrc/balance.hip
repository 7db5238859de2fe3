// A router's balance: choice, weights, counts and loss of a batch of tokens, and the gradient of the logits.
//
// A wave takes a token at a time; lane l holds experts l, l + 64, ...  The sums
// over the tokens are kept by each lane for its experts, added up within the
// workgroup, and over the workgroups, in order, by a second kernel.
#include "balance.h"

namespace ftmoe {

namespace {

constexpr int kWaves = 16;
constexpr float kInf = __builtin_huge_valf();

__device__ __attribute__((always_inline)) inline float wave_max(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
  return v;
}
__device__ __attribute__((always_inline)) inline float wave_sum(float v) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}

// A token's logits, J for each lane; -inf beyond the last.
template <typename X, int J>
struct Logits {
  float z[J];
  __device__ __attribute__((always_inline)) inline void load(const X* row, int experts, int lane) {
#pragma unroll
    for (int j = 0; j < J; ++j) {
      const int e = lane + 64 * j;
      z[j] = e < experts ? float(gload<X>(row + e)) : -kInf;
    }
  }
  // whether some logit is not -inf
  __device__ __attribute__((always_inline)) inline bool some() const {
    bool any = false;
#pragma unroll
    for (int j = 0; j < J; ++j) any = any || !(z[j] == -kInf);
    return __any(any);
  }
  // softmax; 0 beyond the last expert
  __device__ __attribute__((always_inline)) inline void softmax(float (&p)[J], int experts, int lane) const {
    float top = -kInf;
#pragma unroll
    for (int j = 0; j < J; ++j) top = fmaxf(top, z[j]);
    top = wave_max(top);
    float sum = 0.f;
#pragma unroll
    for (int j = 0; j < J; ++j) {
      p[j] = lane + 64 * j < experts ? expf(z[j] - top) : 0.f;
      sum += p[j];
    }
    sum = 1.f / wave_sum(sum);
#pragma unroll
    for (int j = 0; j < J; ++j) p[j] *= sum;
  }
};

template <typename X, int J>
__global__ __launch_bounds__(64 * kWaves) void k_balance(BalanceForward a) {
  __shared__ float lds_p[kWaves][64 * J];
  __shared__ int lds_c[64 * J];
  __shared__ int lds_v;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int e = threadIdx.x; e < 64 * J; e += 64 * kWaves) lds_c[e] = 0;
  if (threadIdx.x == 0) lds_v = 0;
  __syncthreads();
  float sums[J] = {};
  int counted = 0;
  for (int64_t t = int64_t(blockIdx.x) * kWaves + wave; t < a.tokens; t += int64_t(a.groups) * kWaves) {
    Logits<X, J> l;
    l.load(static_cast<const X*>(a.logits) + t * a.ld, a.experts, lane);
    const bool on = (!a.valid || gload<uint8_t>(a.valid + t)) && l.some();
    int mine = -1;          // lane i: the choice of rank i, and its logit
    float mine_z = -kInf, first = 0.f;
    if (on) {
      ++counted;
      float p[J];
      l.softmax(p, a.experts, lane);
#pragma unroll
      for (int j = 0; j < J; ++j) sums[j] += p[j];
      for (int i = 0; i < a.top_k; ++i) {
        float best = -kInf;
#pragma unroll
        for (int j = 0; j < J; ++j) best = fmaxf(best, l.z[j]);  // NaN is passed over
        best = wave_max(best);
        if (best == -kInf) break;
        int at = 0x7FFFFFFF;
#pragma unroll
        for (int j = J - 1; j >= 0; --j) at = l.z[j] == best ? lane + 64 * j : at;
#pragma unroll
        for (int o = 32; o > 0; o >>= 1) at = min(at, __shfl_xor(at, o));
#pragma unroll
        for (int j = 0; j < J; ++j)
          if (lane + 64 * j == at) l.z[j] = -kInf;
        if (i == 0) first = best;
        if (lane == i) {
          mine = at;
          mine_z = best;
        }
      }
      if (mine >= 0) atomicAdd(&lds_c[mine], 1);
    }
    const float ex = mine >= 0 ? expf(mine_z - first) : 0.f;
    const float sum = wave_sum(ex);
    if (lane < a.top_k) {
      a.sel[t * a.top_k + lane] = mine;
      a.w[t * a.top_k + lane] = mine >= 0 ? ex / sum : 0.f;
    }
  }
#pragma unroll
  for (int j = 0; j < J; ++j) lds_p[wave][lane + 64 * j] = sums[j];
  if (lane == 0) atomicAdd(&lds_v, counted);
  __syncthreads();
  for (int e = threadIdx.x; e < a.experts; e += 64 * kWaves) {
    float s = 0.f;
    for (int i = 0; i < kWaves; ++i) s += lds_p[i][e];
    a.part_p[int64_t(blockIdx.x) * a.experts + e] = s;
    a.part_c[int64_t(blockIdx.x) * a.experts + e] = lds_c[e];
  }
  if (threadIdx.x == 0) a.part_v[blockIdx.x] = lds_v;
}

// one workgroup
__global__ __launch_bounds__(512) void k_balance_join(BalanceForward a) {
  __shared__ double lds[512];
  const int e = threadIdx.x;
  double p = 0.0;
  int c = 0, v = 0;
  if (e < a.experts) {
    for (int g = 0; g < a.groups; ++g) {
      p += double(a.part_p[int64_t(g) * a.experts + e]);
      c += a.part_c[int64_t(g) * a.experts + e];
    }
    a.counts[e] = c;
  }
  lds[e] = p * c;
  __syncthreads();
  if (e == 0) {
    for (int g = 0; g < a.groups; ++g) v += a.part_v[g];
    a.counts[a.experts] = v;
    double sum = 0.0;
    for (int i = 0; i < a.experts; ++i) sum += lds[i];
    const double n = double(v);
    a.loss[0] = v ? float(double(a.weight) * a.experts / (a.top_k * n * n) * sum) : 0.f;
  }
}

template <typename X, int J>
__global__ __launch_bounds__(64 * kWaves) void k_balance_backward(BalanceBackward a) {
  __shared__ float lds[kWaves][64 * J];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
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
  for (int64_t t = int64_t(blockIdx.x) * kWaves + wave; t < a.tokens; t += int64_t(gridDim.x) * kWaves) {
    Logits<X, J> l;
    l.load(static_cast<const X*>(a.logits) + t * a.ld, a.experts, lane);
    X* dz = static_cast<X*>(a.dlogits) + t * a.ld;
    const bool on = (!a.valid || gload<uint8_t>(a.valid + t)) && l.some();
    float d[J] = {};
    if (on) {
      float p[J], sum = 0.f;
      l.softmax(p, a.experts, lane);
#pragma unroll
      for (int j = 0; j < J; ++j) sum = fmaf(p[j], c[j], sum);
      sum = wave_sum(sum);
#pragma unroll
      for (int j = 0; j < J; ++j) d[j] = dloss * p[j] * (c[j] - sum);
      if (a.dw) {
        const int i = lane < a.top_k ? a.sel[t * a.top_k + lane] : -1;
        const bool chosen = uint32_t(i) < uint32_t(a.experts);
        const float w = chosen ? a.w[t * a.top_k + lane] : 0.f, dw = chosen ? a.dw[t * a.top_k + lane] : 0.f;
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
  hipLaunchKernelGGL((k_balance<X, J>), dim3(uint32_t(a.groups)), dim3(64 * kWaves), 0, s, a);
  hipLaunchKernelGGL(k_balance_join, dim3(1), dim3(512), 0, s, a);
  return hipGetLastError();
}
template <typename X, int J>
hipError_t launch(const BalanceBackward& a, hipStream_t s) {
  const uint32_t grid = uint32_t(balance_groups(a.tokens));
  hipLaunchKernelGGL((k_balance_backward<X, J>), dim3(grid), dim3(64 * kWaves), 0, s, a);
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
  const int32_t g = (tokens + kWaves - 1) / kWaves;
  return g < 1 ? 1 : g < 256 ? g : 256;
}

hipError_t launch_balance(int dtype, const BalanceForward& a, hipStream_t s) { return launch_type(dtype, a, s); }
hipError_t launch_balance_backward(int dtype, const BalanceBackward& a, hipStream_t s) {
  return launch_type(dtype, a, s);
}

}  // namespace ftmoe
