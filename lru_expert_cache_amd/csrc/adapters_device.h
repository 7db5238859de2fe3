// Device side of the adapters: tiles, and rows of either product.
#pragma once
#include <algorithm>

#include "adapters.h"
#include "dense.h"

namespace ftmoe {

// A tile as a wave sees it: lane l has tokens l % 16, + 16, ... of it; beyond the last, the last again.
template <int SUB>
struct TileTokens {
  int id, count;
  int token[SUB];
  bool live;
};

// Tile `item` of up to 64 tokens: the wave holds a token's id in each lane and
// counts, for each token, those of the same adapter before it; every 16th of
// an adapter begins a tile.
__device__ __attribute__((always_inline)) inline TileTokens<1> few_tile(const Adapters& l, int item) {
  const int lane = threadIdx.x & 63;
  int group = -1;
  if (lane < l.tokens) {
    const int id = gload<int32_t>(l.ids + lane);
    group = uint32_t(id) < uint32_t(l.count) ? id : l.in_place ? -1 : l.count;
  }
  int rank = 0;
  for (int j = 0; j < l.tokens; ++j) {
    const int other = __builtin_amdgcn_readlane(group, j);
    rank += (other == group) & (j < lane);
  }
  const bool start = group >= 0 && rank % 16 == 0;
  const uint64_t starts = __ballot(start);
  const int nth = __popcll(starts & ((uint64_t(1) << lane) - 1));
  TileTokens<1> t{};
  t.live = item < __popcll(starts);
  if (!t.live) return t;
  const int src = __builtin_ctzll(__ballot(start && nth == item));
  t.id = __builtin_amdgcn_readlane(group, src);
  const int first = __builtin_amdgcn_readlane(rank, src);
  const bool mine = group == t.id && rank >= first && rank < first + 16;
  t.count = __popcll(__ballot(mine));
  // each of its lanes sends its number to the lane of its place (the others to one that nobody reads)
  const int token = __builtin_amdgcn_ds_permute((mine ? rank - first : 63) * 4, lane);
  t.token[0] = __builtin_amdgcn_ds_bpermute(min(lane % 16, t.count - 1) * 4, token);
  return t;
}

template <int SUB>
__device__ __attribute__((always_inline)) inline TileTokens<SUB> find_tile(const Adapters& l, uint32_t item) {
  TileTokens<SUB> t{};
  if constexpr (SUB == 1)
    if (l.few) return few_tile(l, int(item));
  const uint32_t window = l.by_cap(item);
  t.live = int(item - window * uint32_t(l.tile_cap)) < gload<int32_t>(l.tile_count + window);
  if (!t.live) return t;
  static_assert(sizeof(AdapterTile) == 16, "one load");
  const u32x4 w = gload<u32x4>(l.tiles + item);  // id, first, count
  t.id = __builtin_amdgcn_readfirstlane(int(w[0]));
  t.count = __builtin_amdgcn_readfirstlane(int(w[2]));
#pragma unroll
  for (int m = 0; m < SUB; ++m)
    t.token[m] = gload<int32_t>(l.order + int(w[1]) + min(int(threadIdx.x & 15) + 16 * m, t.count - 1));
  return t;
}

// Workgroups are handed to the eight XCDs in turn; each takes a range of the
// work next to each other, so that tiles of one adapter find its matrices in
// their XCD's cache.  Rounds of the loop go over adapter_rounds(total) numbers.
constexpr uint32_t kXcds = 8;
__host__ __device__ inline uint32_t adapter_rounds(uint32_t total) { return (total + kXcds - 1) / kXcds * kXcds; }
__device__ __attribute__((always_inline)) inline uint32_t adapter_work(uint32_t round, uint32_t total) {
  return round % kXcds * (adapter_rounds(total) / kXcds) + round / kXcds;
}
// workgroups of a launch, which go on to further rounds if there are more (a multiple of the XCDs)
inline uint32_t adapter_grid(uint32_t total) { return std::min(adapter_rounds(total), uint32_t(1) << 22); }

// Eight neighbouring elements of a row of `width`, as a matrix instruction
// takes them, from element 8 c.  Where the row ends within them, or before,
// its last eight are taken instead: the places that are another piece's
// (those below 8 c) are zeros in one operand (ZERO), so that the products are
// those of the row, and nothing outside it is read.  Loops that are not
// unrolled keep the code short: what a cold start fetches of it counts.
template <typename E, bool ZERO>
__device__ __attribute__((always_inline)) inline u32x4 row_piece(const E* row, int c, int width) {
  typedef u32x4 __attribute__((aligned(1))) any;
  typedef uint64_t u64x2 __attribute__((ext_vector_type(2)));
  if (width >= 8) {
    const int from = min(8 * c, width - 8);
    const u32x4 v = gload<any>(row + from);
    if constexpr (!ZERO) return v;
    u64x2 w = (u64x2)v;
    const int skip = 8 * c - from;  // elements
    const int lo = 16 * min(skip, 4), hi = 16 * min(max(skip - 4, 0), 4);
    w[0] = lo == 64 ? 0 : w[0] >> lo << lo;
    w[1] = hi == 64 ? 0 : w[1] >> hi << hi;
    return (u32x4)w;
  }
  u64x2 w{};
#pragma nounroll
  for (int i = width - 1 - 8 * c; i >= 0; --i) {
    w[1] = w[1] << 16 | w[0] >> 48;
    w[0] = w[0] << 16 | __builtin_bit_cast(uint16_t, gload<E>(row + 8 * c + i));
  }
  return (u32x4)w;
}

}  // namespace ftmoe
