// How a call of the adapters is cut: a rule on sizes.
#include <algorithm>

#include "adapters.h"

namespace ftmoe {

AdapterPlan adapter_plan(int32_t tokens, int32_t in, int32_t out, int32_t rank, int32_t count, int base_bytes,
                         int out_bytes) {
  AdapterPlan p{};
  const int32_t most = std::min(tokens, kAdapterWindow);
  p.few = tokens <= kAdapterFew;
  p.sub = 1;
  // Larger tiles read an adapter's matrices less often and leave more places
  // empty.  Tiles of 16, 32 and 64 tokens, prompts, bf16, us: 512 tokens (in =
  // out = 7168, rank 64) 26 / 25 / 29; 2048 tokens (2048, rank 16) 22 / 20 /
  // 22; 8192 tokens (2048, rank 64) 71 / 58 / 58; 8192 tokens (7168, rank 64)
  // 194 / 137 / 115; 1531 tokens (rank 8, a quarter of them single) 29 / 35 /
  // -; rank 128, 8192 tokens: 320 / 189 / -.  The host knows the table's size alone, and takes every adapter in it to be
  // asked for: 8192 tokens (7168, rank 64) of 16 adapters in a table of 16 / 129 / 257 / 1024: 110 / 134 / 179 / 167 us.
  if (rank <= 128 && int64_t(tokens) * (rank > 16 ? 2 : 1) >= 2048 && tokens >= 32 * count) p.sub = 2;
  if (rank <= 64 && tokens >= 4096 && int64_t(in) + out >= 8192 && tokens >= 64 * count) p.sub = 4;
  p.windows = std::max(1, (tokens + kAdapterWindow - 1) / kAdapterWindow);
  // each adapter (and the tokens that have none) can leave one tile partly filled
  p.tile_cap = int32_t(std::min<int64_t>(most, most / (16 * p.sub) + int64_t(count) + 1));
  // About a workgroup on each CU, so that none waits for a second round (8192
  // tokens, 7168, rank 64: 42 us with two parts, 52 with three, 43 with four);
  // 256 elements of K a part at least.  Half of the adapters are taken to have a last tile partly filled.
  const int64_t rows = (rank + 63) / 64;
  const int64_t tiles = int64_t(p.windows) * std::min<int64_t>(p.tile_cap, tokens / (16 * p.sub) + 1 + count / 2) * rows;
  p.parts = int32_t(std::clamp<int64_t>(std::min<int64_t>((256 + tiles / 2) / tiles, in / 256), 1, 32));
  // One launch where a workgroup soon has all of A x: graphs of calls (rank 16, N 4096), one launch against two, us:
  // one / 8 / 32 tokens of as many adapters, K 2560: 6.6 / 8.0 / 8.4 against 7.4 / 8.3 / 8.9; 3584: 7.2 / 9.3 / 9.8
  // against 7.5 / 8.7 / 9.4.  Calls by themselves save up to the launch's 2 us too.  The width alone decides, for any
  // number of tokens: one alone would still gain 0.3 us at 3584, where 8 and 32 lose 0.6 and 0.4.  Ranks above 16 have
  // no such kernel (one token, rank 64, 2048 / 6144: 9.3 / 8.5 us in two launches).
  p.once = p.few && rank <= 16 && in <= 2560;
  p.out_step = 32 * (p.once ? 16 : 4 * adapter_out_blocks(base_bytes, out_bytes, p.sub, rank));
  // columns for about 1024 workgroups: each joins h's parts first (8192 tokens, 7168, rank 64: steps of 256 columns
  // 1 / 2 / 4 / 7 a workgroup: 132 / 118 / 115 / 128 us for the call); for fewer where each forms h itself (64 tokens
  // of 64 adapters, 2048 into 16384: 14.9 us, in 1024 workgroups 18.9).  Few tokens are taken to be of as many adapters.
  const int64_t blocks = (out + p.out_step - 1) / p.out_step;
  const int64_t each = p.few ? p.tile_cap * rows : tiles, goal = p.once ? 448 : 1024;
  p.out_blocks = int32_t(std::clamp<int64_t>((blocks * each + goal / 2) / goal, 1, 8));
  // (numbers of workgroups stay below 2^30)
  const int64_t all = int64_t(p.windows) * p.tile_cap;
  p.out_blocks = int32_t(std::max<int64_t>(p.out_blocks, (all * blocks >> 30) + 1));
  return p;
}

}  // namespace ftmoe
