// Low-rank adapters beside a projection, token by token.
#include "adapters.h"

namespace ftmoe {

namespace {

// h[t][r] = sum_k A[i][r][k] x[t][k]: a wave for each sum
template <typename E>
__global__ __launch_bounds__(256) void k_adapters_in(Adapters l) {
  const int64_t t = blockIdx.x;
  const int id = l.ids[t];
  if (uint32_t(id) >= uint32_t(l.count)) return;
  const int lane = threadIdx.x & 63;
  const E* x = static_cast<const E*>(l.x) + t * l.ld_x;
  for (int r = threadIdx.x >> 6; r < l.rank; r += 4) {
    const E* a = static_cast<const E*>(l.a) + (int64_t(id) * l.rank + r) * l.ld_a;
    float sum = 0.f;
    for (int k = lane; k < l.in; k += 64) sum = fmaf(float(gload<E>(a + k)), float(gload<E>(x + k)), sum);
#pragma unroll
    for (int o = 32; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
    if (lane == 0) l.h[t * l.rank + r] = sum;
  }
}

// y[t][n] = base[t][n] + scale[i] sum_r B[i][n][r] h[t][r]: a thread for each
template <typename E, typename B, typename Y>
__global__ __launch_bounds__(256) void k_adapters_out(Adapters l) {
  const int64_t t = blockIdx.x;
  const int n = int(blockIdx.y) * 256 + int(threadIdx.x);
  if (n >= l.out) return;
  const int id = l.ids[t];
  const bool on = uint32_t(id) < uint32_t(l.count);
  if (!on && l.in_place) return;
  float sum = 0.f;
  if (on) {
    const E* b = static_cast<const E*>(l.b) + (int64_t(id) * l.out + n) * l.ld_b;
    for (int r = 0; r < l.rank; ++r) sum = fmaf(float(gload<E>(b + r)), l.h[t * l.rank + r], sum);
    if (l.scale) sum *= l.scale[id];
  }
  if (l.base) sum += float(gload<B>(static_cast<const B*>(l.base) + t * l.ld_base + n));
  gstore<Y>(static_cast<Y*>(l.y) + t * l.ld_y + n, Y(sum));
}

template <typename E>
hipError_t launch(int base_dtype, int out_dtype, const Adapters& l, hipStream_t s) {
  hipLaunchKernelGGL((k_adapters_in<E>), dim3(uint32_t(l.tokens)), dim3(256), 0, s, l);
  const dim3 grid(uint32_t(l.tokens), uint32_t((l.out + 255) / 256));
  if (out_dtype == FT_DT_F32)
    hipLaunchKernelGGL((k_adapters_out<E, float, float>), grid, dim3(256), 0, s, l);
  else if (base_dtype == FT_DT_F32)
    hipLaunchKernelGGL((k_adapters_out<E, float, E>), grid, dim3(256), 0, s, l);
  else
    hipLaunchKernelGGL((k_adapters_out<E, E, E>), grid, dim3(256), 0, s, l);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_adapters(int dtype, int base_dtype, int out_dtype, const Adapters& l, hipStream_t s) {
  return dtype == FT_DT_F16 ? launch<_Float16>(base_dtype, out_dtype, l, s) : launch<__bf16>(base_dtype, out_dtype, l, s);
}

}  // namespace ftmoe
