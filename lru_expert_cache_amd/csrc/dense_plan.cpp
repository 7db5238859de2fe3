// Which kernel runs a dense product, and how: rules on sizes, strides and
// alignment alone, so that the scratch memory a call needs is known before it.
#include <algorithm>

#include "dense.h"

namespace ftmoe {

namespace {

int64_t parts(int64_t v, int64_t by) { return (v + by - 1) / by; }
bool on16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

}  // namespace

// The tiled kernels load whole 16-byte pieces and hold a unit's offsets in 31
// bits: 128 rows of an operand along K, 64 (8 bit: 128) of one across it.
bool dense_tileable(DenseForm form, const DenseProblem& p) {
  const int64_t es = dense_elem(form);
  if (!on16(p.a[0]) || !on16(p.a[1]) || !on16(p.b[0]) || !on16(p.b[1]) || p.lda % 16 || p.ldb % 16) return false;
  if (p.lda >= (1 << 23) || p.ldb >= (1 << 23)) return false;
  if ((dense_a_rows(form) || dense_b_rows(form)) && int64_t(p.k) * es % 16) return false;
  if (!dense_a_rows(form) && int64_t(p.m) * es % 16) return false;
  if (!dense_b_rows(form) && int64_t(p.n) * es % 16) return false;
  return true;
}

int64_t dense_part_bytes(DenseForm form, const DenseShape& s, int splits) {
  if (splits <= 1) return 0;
  return int64_t(splits) * (dense_two_b(form) ? 2 : 1) * s.m * parts(s.n, 4) * 16;
}

// Estimated times in microseconds.  A 256 x 256 workgroup has a CU to itself
// and takes kStep256 per K step; 128 x 128 ones run two to a CU, kStep128 a
// step when two share it and kStep128Alone when not.  Cutting K costs a second
// launch and the parts' way to memory and back.
DensePlan dense_plan(DenseForm form, const DenseShape* shapes, int count) {
  constexpr double kStep256 = 1.65, kStep128 = 1.05, kStep128Alone = 0.65, kStart = 2.5, kJoin = 3.0, kBytes = 4e6;
  constexpr int kCus = 256, kMaxSplits = 32;
  const int ke = 128 / dense_elem(form);
  DensePlan best{128, 1};
  double best_t = 1e30;
  for (int tile : {256, 128}) {
    int64_t tiles = 0, steps = 0, bytes = 0;
    for (int i = 0; i < count; ++i) {
      const DenseShape& s = shapes[i];
      tiles += parts(s.m, tile) * parts(s.n, dense_two_b(form) ? tile / 2 : tile);
      steps = std::max(steps, parts(s.k, ke) * s.segs);
      bytes += dense_part_bytes(form, s, 2) / 2;
    }
    for (int splits = 1; splits <= kMaxSplits && splits <= std::max<int64_t>(1, steps / 2); ++splits) {
      const int64_t wgs = tiles * splits, per = parts(steps, splits);
      double t;
      if (tile == 256) {
        t = double(parts(wgs, kCus)) * (kStart + per * kStep256);
      } else {
        const int64_t full = wgs / (2 * kCus), rest = wgs % (2 * kCus);
        t = double(full) * (kStart + per * kStep128);
        if (rest) t += kStart + per * (rest > kCus ? kStep128 : kStep128Alone);
      }
      if (splits > 1) t += kJoin + double(splits) * 2 * double(bytes) / kBytes;
      if (t < best_t) best_t = t, best = {tile, splits};
    }
  }
  return best;
}

hipError_t launch_dense_tile(DenseForm form, int dtype, int tile, const DenseLaunch& l, hipStream_t s) {
  if (dense_int(form)) return launch_dense_tile_int(form, dtype, tile, l, s);
  return dtype == FT_DT_F16 ? launch_dense_tile_f16(form, tile, l, s) : launch_dense_tile_bf16(form, tile, l, s);
}

}  // namespace ftmoe
