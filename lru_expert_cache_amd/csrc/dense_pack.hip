// Operands whose rows are not whole 16-byte pieces at 16-byte distances, copied
// into rows that are, zeros behind them: the tiled kernels then take them.
//
// One launch for all of a call's copies; a thread writes 16 bytes at a time,
// read with one unaligned load where the source has them.  Bound by HBM: a
// weight matrix is read and written once, which costs less than the general
// kernel loses from 1 token on (8-bit block of 8 tokens, H 2417, I 1984: 81 us
// on the general kernel, 24 us with the copies; bf16 backward of 4000 tokens, H 2721,
// I 1043: 978 and 216 us).
#include "dense.h"

namespace ftmoe {

namespace {

// 2^lanes[y] threads take a row of copy y
__global__ __launch_bounds__(256) void k_dense_pack(DensePackLaunch l) {
  const DensePack& p = l.p[blockIdx.y];
  const int lanes = 1 << p.lanes, per = 256 >> p.lanes;
  const int64_t pieces = p.dst_bytes / 16;
  for (int64_t row = int64_t(blockIdx.x) * per + (int(threadIdx.x) >> p.lanes); row < p.rows; row += int64_t(gridDim.x) * per)
    for (int64_t i = int(threadIdx.x) & (lanes - 1); i < pieces; i += lanes) {
      const uint8_t* s = p.src + row * p.src_ld + i * 16;
      const int64_t have = p.bytes - i * 16;
      u32x4 v = {0, 0, 0, 0};
      if (have >= 16) {
        typedef u32x4 __attribute__((aligned(1))) any;
        v = gload<any>(s);
      } else if (have > 0) {
        uint8_t b[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) b[j] = j < have ? gload<uint8_t>(s + j) : uint8_t(0);
        __builtin_memcpy(&v, b, 16);
      }
      gstore<u32x4>(p.dst + row * p.dst_ld + i * 16, v);
    }
}

}  // namespace

hipError_t launch_dense_pack(const DensePackLaunch& packs, hipStream_t s) {
  constexpr int64_t kMost = 2048;  // workgroups of a copy: the card eight times over
  DensePackLaunch l = packs;
  int64_t wgs = 0;
  for (int i = 0; i < l.count; ++i) {
    DensePack& p = l.p[i];
    p.lanes = 0;
    while (p.lanes < 8 && (int64_t(16) << p.lanes) < p.dst_bytes) ++p.lanes;
    const int64_t per = 256 >> p.lanes, n = (p.rows + per - 1) / per;
    wgs = n > wgs ? n : wgs;
  }
  if (wgs == 0) return hipSuccess;
  hipLaunchKernelGGL(k_dense_pack, dim3(uint32_t(wgs < kMost ? wgs : kMost), l.count), dim3(256), 0, s, l);
  return hipGetLastError();
}

}  // namespace ftmoe
