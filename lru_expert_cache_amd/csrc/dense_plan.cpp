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

// Estimated times in microseconds, fitted to sweeps of tiles and parts over 10
// sizes of each form.  A 256 x 256 workgroup has a CU to itself; a K step takes
// it longer the more CUs are busy (they share power and the L2s).  128 x 128
// ones run two to a CU, and read the operands twice as often: slower than 256
// x 256 once the card is at its power limit (8192^3: 1025 us against 838), but
// quicker where they fill the CUs better (1531 x 7168 x 2048: 46 against 50;
// 4096 x 2048 x 768: 18.6 against 26.5).  Cutting K costs a second launch and
// the parts' way to memory and back (77 x 2048 into 768: 23 us in one part,
// 11 in eight; 4096 x 768 into 2048: 18.6 in one, 39 in two).
DensePlan dense_plan(DenseForm form, const DenseShape* shapes, int count) {
  constexpr int kCus = 256, kMaxSplits = 32;
  constexpr double kStart = 4.0, kJoin = 5.0, kJoinBytes = 3.5e6;  // bytes of a part per us, written and read
  const bool i8 = dense_int(form);
  // a step of a 256 x 256 tile with few and with all CUs busy; of a 128 x 128
  // one alone on its CU likewise, of a pair of them, and of a pair at the power
  // limit; what a tile takes beside its steps
  const double few256 = i8 ? 1.0 : 1.15, all256 = i8 ? 1.35 : 1.55, tile256 = i8 ? 9.0 : 3.0;
  const double few128 = 0.36, all128 = i8 ? 0.6 : 0.52, pair128 = i8 ? 0.9 : 0.75, hot128 = i8 ? 1.1 : 1.0, tile128 = 1.5;
  const double epilogue = form == kDenseGrad ? 6.0 : 0.0;  // its reads of gu, in one part
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
    const int most = int(std::min<int64_t>(kMaxSplits, std::max<int64_t>(1, steps / 2)));
    for (int splits = 1; splits <= most; ++splits) {
      const int64_t wgs = tiles * splits, per = parts(steps, splits);
      const double busy = std::min(1.0, double(wgs) / kCus);
      const int64_t each = parts(wgs, kCus);  // a CU's tiles
      double t = kStart;
      if (tile == 256) {
        t += double(each) * (tile256 + per * (few256 + (all256 - few256) * busy));
      } else {
        t += double(each / 2) * (tile128 + per * (each <= 8 ? pair128 : hot128));
        if (each % 2) t += tile128 + per * (few128 + (all128 - few128) * busy);
      }
      t += splits > 1 ? kJoin + double(splits) * double(bytes) / kJoinBytes : epilogue;
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
