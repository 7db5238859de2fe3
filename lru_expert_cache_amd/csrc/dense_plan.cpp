// Which kernel runs a dense product, and how: rules on sizes, strides and
// alignment alone, so that the scratch memory a call needs is known before it.
#include <algorithm>

#include "dense.h"

namespace ftmoe {

namespace {

int64_t parts(int64_t v, int64_t by) { return (v + by - 1) / by; }
bool on16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

}  // namespace

// The tiled kernels load whole 16-byte pieces (a piece that K or the columns
// end in has to be there, with zeros) and hold a unit's offsets in 31 bits: 128
// rows of an operand along K, 64 (8 bit: 128) of one across it.
bool dense_tileable(DenseForm form, const DenseProblem& p) {
  const int64_t es = dense_elem(form);
  if (!on16(p.a[0]) || !on16(p.a[1]) || !on16(p.b[0]) || !on16(p.b[1]) || p.lda % 16 || p.ldb % 16) return false;
  if (p.lda >= (1 << 23) || p.ldb >= (1 << 23)) return false;
  if ((dense_a_rows(form) ? p.k : p.m) * es % 16 && !p.a_whole) return false;
  if ((dense_b_rows(form) ? p.k : p.n) * es % 16 && !p.b_whole) return false;
  return true;
}

int64_t dense_part_bytes(DenseForm form, const DenseShape& s, int splits) {
  if (splits <= 1) return 0;
  return int64_t(splits) * (dense_two_b(form) ? 2 : 1) * s.m * parts(s.n, 4) * 16;
}

// Estimated times in microseconds, fitted to 37 products and blocks of normal
// random numbers, each with either tile alone: within 13% of 71 of the 74 times
// (three products of 300 to 1500 tokens with K in parts come out a fifth low).
// The choice is within 1% of the better tile, where the two launches of a block
// take different ones within 6% of the better of one tile for both.  A 256 x 256 workgroup has a CU to itself, 128 x 128
// ones run two to a CU and read the operands twice as often; a K step takes
// longer the more of the card's places are taken over the launch, which shares
// power and the L2s.  So 256 x 256 is quicker where
// it fills the card (forward of 8192 tokens, H 7168, I 2048: 530 us against
// 696; 8-bit 4096 x 6144 x 6144 131 against 142), 128 x 128 where it does that
// better (4096 tokens, H 2048, I 768: 45 against 64; 8-bit 1024 x 6144 x 6144 48
// against 62).  Cutting K costs a second launch and
// the parts' way to memory and back (77 x 2048 into 768: 23 us in one part,
// 11 in eight; 4096 x 768 into 2048: 18.6 in one, 39 in two).
namespace {

constexpr int kCus = 256;
constexpr double kStart = 4.0;

// a tile beside its steps, and a step with few and with all places of the card taken
struct Pace {
  double tile256, few256, all256;
  double tile128, few128, all128;  // alone on its CU
  double few2, all2;               // two on a CU, each
};
Pace pace(DenseForm form) {
  return dense_int(form) ? Pace{5.5, 0.87, 1.46, 0.7, 0.36, 0.5, 0.43, 1.06} : Pace{5.3, 0.8, 1.41, 0.6, 0.34, 0.56, 0.39, 0.97};
}
double between(double few, double all, double taken) { return few + (all - few) * std::min(1.0, taken); }

int64_t tiles_of(DenseForm form, const DenseShape& s, int tile) {
  return parts(s.m, tile) * parts(s.n, dense_two_b(form) ? tile / 2 : tile);
}
int64_t steps_of(DenseForm form, const DenseShape& s) { return parts(s.k, 128 / dense_elem(form)) * s.segs; }

// wgs workgroups of `per` steps each
double tiles_time(DenseForm form, int tile, int64_t wgs, int64_t per) {
  const Pace p = pace(form);
  if (tile == 256) {
    const int64_t each = parts(wgs, kCus);
    return kStart + double(each) * (p.tile256 + per * between(p.few256, p.all256, double(wgs) / double(each * kCus)));
  }
  // rounds of two a CU, the last one of one where that holds the rest
  const int64_t whole = wgs / (2 * kCus), rest = wgs % (2 * kCus);
  const double taken = double(rest) / kCus;
  double t = kStart + double(whole) * (p.tile128 + per * p.all2);
  if (rest) t += p.tile128 + per * (rest <= kCus ? between(p.few128, p.all128, taken) : between(p.few2, p.all2, taken / 2));
  return t;
}

DensePlan plan_of(DenseForm form, const DenseShape* shapes, int count, double* time) {
  constexpr int kMaxSplits = 32;
  constexpr double kJoin = 5.0, kJoinBytes = 3.5e6;  // bytes of a part per us, written and read
  const double epilogue = form == kDenseGrad ? 6.0 : 0.0;  // its reads of gu, in one part
  DensePlan best{128, 1};
  *time = 1e30;
  for (int tile : {256, 128}) {
    int64_t tiles = 0, steps = 0, bytes = 0;
    int32_t rows = 0;
    for (int i = 0; i < count; ++i) {
      rows = std::max(rows, shapes[i].m);
      tiles += tiles_of(form, shapes[i], tile);
      steps = std::max(steps, steps_of(form, shapes[i]));
      bytes += dense_part_bytes(form, shapes[i], 2) / 2;
    }
    // half of each tile would stay empty (the fit gives such products 128 x 128 anyway; few tokens
    // whose rests fill the half have no other kernel)
    if (tile == 256 && rows <= 128) continue;
    // more parts than fill the card a few times over only cost their way to memory
    const int64_t useful = 1 + parts(4 * kCus, std::max<int64_t>(1, tiles));
    const int most = int(std::min({int64_t(kMaxSplits), useful, std::max<int64_t>(1, steps / 2)}));
    for (int splits = 1; splits <= most; ++splits) {
      double t = tiles_time(form, tile, tiles * splits, parts(steps, splits));
      t += splits > 1 ? kJoin + double(splits) * double(bytes) / kJoinBytes : epilogue;
      if (t < *time) *time = t, best = {tile, splits};
    }
  }
  return best;
}

}  // namespace

DensePlan dense_plan(DenseForm form, const DenseShape* shapes, int count) {
  double t;
  return plan_of(form, shapes, count, &t);
}

// One queue of both keeps the CUs busy to the end: its time is the work over
// the places, but at least one longest tile.  Only products that are not cut
// alone either are run so: what a gradient comes to does not depend on which
// others are asked for.
int dense_plan_pair(const DenseShape (&outer)[3], const DenseShape& cols, bool only128) {
  double apart_outer, apart_cols;
  if (plan_of(kDenseOuter, outer, 3, &apart_outer).splits != 1 ||
      plan_of(kDenseCols, &cols, 1, &apart_cols).splits != 1)
    return 0;
  int best = 0;
  double best_t = apart_outer + apart_cols;
  const Pace p = pace(kDenseOuter);
  for (int tile : {256, 128}) {
    if (tile == 256 && only128) continue;
    int64_t wgs = 0, work = 0, longest = 0;
    auto add = [&](DenseForm form, const DenseShape& s) {
      const int64_t n = tiles_of(form, s, tile), steps = std::max<int64_t>(2, steps_of(form, s));
      wgs += n;
      work += n * steps;
      if (n) longest = std::max(longest, steps);
    };
    for (const DenseShape& s : outer) add(kDenseOuter, s);
    add(kDenseCols, cols);
    const double over = tile == 256 ? p.tile256 : p.tile128;
    const int places = tile == 256 ? kCus : 2 * kCus;
    const double taken = double(wgs) / places;
    const double alone = tile == 256 ? between(p.few256, p.all256, taken) : between(p.few128, p.all128, 2 * taken);
    const double all = tile == 256 ? alone : between(p.few2, p.all2, taken);
    // the end is uneven by part of a tile of dx, which come last
    const double end = wgs > places ? steps_of(kDenseCols, cols) * all / 4 : 0.0;
    const double t = kStart + std::max(over + longest * alone, (double(work) * all + double(wgs) * over) / places + end);
    if (t < best_t) best_t = t, best = tile;
  }
  return best;
}

hipError_t launch_dense_pair(int dtype, int tile, const DensePair& l, hipStream_t s) {
  return dtype == FT_DT_F16 ? launch_dense_pair_f16(tile, l, s) : launch_dense_pair_bf16(tile, l, s);
}

hipError_t launch_dense_tile(DenseForm form, int dtype, int tile, const DenseLaunch& l, hipStream_t s) {
  if (dense_int(form)) return launch_dense_tile_int(form, dtype, tile, l, s);
  return dtype == FT_DT_F16 ? launch_dense_tile_f16(form, tile, l, s) : launch_dense_tile_bf16(form, tile, l, s);
}

}  // namespace ftmoe
