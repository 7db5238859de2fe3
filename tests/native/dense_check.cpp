// What the dense operators' host code decides, without a GPU (linked against
// the built library):
//   dense_check plan <form> <m n k segs>...   tile and parts of a product, or of up to three of one form
//   dense_check pair <m n k> x 4              the tile of three weight gradients and dx in one launch, or 0
//   dense_check few <form> <tokens>           what the few-token launch makes of tokens of a type (FT_DT_*) yet to
//                                             be quantised: "refused", or "taken"
#include <cstdio>
#include <cstdlib>
#include <cstring>

#include "dense.h"

using namespace ftmoe;

int main(int argc, char** argv) {
  auto arg = [&](int i) { return i < argc ? std::atoi(argv[i]) : 0; };
  if (argc < 3) return 2;
  if (!std::strcmp(argv[1], "plan")) {
    DenseShape s[kDenseMaxProblems];
    const int count = (argc - 3) / 4;
    if (count < 1 || count > kDenseMaxProblems) return 2;
    for (int i = 0; i < count; ++i) s[i] = {arg(3 + 4 * i), arg(4 + 4 * i), arg(5 + 4 * i), arg(6 + 4 * i)};
    const DensePlan p = dense_plan(DenseForm(arg(2)), s, count);
    std::printf("%d %d\n", p.tile, p.splits);
  } else if (!std::strcmp(argv[1], "pair")) {
    DenseShape s[4];
    for (int i = 0; i < 4; ++i) s[i] = {arg(2 + 3 * i), arg(3 + 3 * i), arg(4 + 3 * i), i == 3 ? 2 : 1};
    const DenseShape outer[3] = {s[0], s[1], s[2]};
    std::printf("%d\n", dense_plan_pair(outer, s[3]));
  } else if (!std::strcmp(argv[1], "few")) {
    DenseLaunch l{};
    l.count = l.splits = 1;
    l.p[0].m = 1;  // n is 0: a launch has no workgroup
    l.p[0].tokens = arg(3);
    const hipError_t e = launch_dense_few(DenseForm(arg(2)), FT_DT_F32, l, nullptr);
    std::printf("%s\n", e == hipErrorInvalidValue ? "refused" : "taken");
  } else {
    return 2;
  }
  return 0;
}
