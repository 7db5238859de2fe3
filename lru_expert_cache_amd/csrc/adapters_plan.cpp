// How a call of the adapters is cut: a rule on sizes.
#include <algorithm>

#include "adapters.h"

namespace ftmoe {

AdapterPlan adapter_plan(int32_t tokens, int32_t in, int32_t out, int32_t rank, int32_t count) {
  AdapterPlan p{};
  const int32_t most = std::min(tokens, kAdapterWindow);
  p.few = tokens <= kAdapterFew;
  p.sub = 1;
  // larger tiles read an adapter's matrices less often, once an adapter has that many tokens
  if (rank <= 64 && tokens / 64 >= 4 * count) p.sub = 4;
  else if (rank <= 64 && tokens / 32 >= 4 * count) p.sub = 2;
  p.windows = std::max(1, (tokens + kAdapterWindow - 1) / kAdapterWindow);
  // each adapter (and the tokens that have none) can leave one tile partly filled
  p.tile_cap = int32_t(std::min<int64_t>(most, most / (16 * p.sub) + int64_t(count) + 1));
  // about two workgroups on each CU; 256 elements of K a part at least
  const int64_t rows = p.sub == 1 && rank > 64 ? (rank + 63) / 64 : 1;
  const int64_t tiles = int64_t(p.windows) * std::min<int64_t>(p.tile_cap, tokens / (16 * p.sub) + 1 + count / 2) * rows;
  p.parts = int32_t(std::clamp<int64_t>(std::min<int64_t>(512 / tiles, in / 256), 1, 32));
  const int64_t blocks = (out + 127) / 128;  // of a workgroup's 128 columns
  p.out_blocks = int32_t(std::clamp<int64_t>(blocks * tiles / 1024, 1, 8));
  // (numbers of workgroups stay below 2^30)
  const int64_t all = int64_t(p.windows) * p.tile_cap;
  p.out_blocks = int32_t(std::max<int64_t>(p.out_blocks, (all * blocks >> 30) + 1));
  return p;
}

}  // namespace ftmoe
