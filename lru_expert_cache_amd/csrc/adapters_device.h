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
};

// Workgroups are handed to the eight XCDs in turn; each XCD takes a range of a
// window's pieces of work next to each other, so that the tiles of one adapter
// find its matrices in their XCD's cache.  The piece of workgroup (or round)
// `at` of a window with `pieces`, or one that is not there.
constexpr uint32_t kXcds = 8;
__device__ __attribute__((always_inline)) inline uint32_t xcd_piece(uint32_t at, uint32_t pieces) {
  const uint32_t per = (pieces + kXcds - 1) / kXcds;
  return at / kXcds < per ? at % kXcds * per + at / kXcds : pieces;
}

// The tile of round `at` among up to 64 tokens, and which of its `each` pieces
// of work.  The wave holds a token's id in each lane and counts, for each
// token, those of the same adapter before it; every 16th begins a tile.
__device__ __attribute__((always_inline)) inline bool few_tile(const Adapters& l, uint32_t at, FastDiv each, bool bare,
                                                               TileTokens<1>& t, int& piece) {
  const int lane = threadIdx.x & 63;
  int group = -1;
  if (lane < l.tokens) {
    const int id = gload<int32_t>(l.ids + lane);
    group = uint32_t(id) < uint32_t(l.count) ? id : bare && !l.in_place ? l.count : -1;
  }
  // lanes of the same adapter, bit by bit of its number (13 bits, those of "none" all ones): a comparison with one
  // token after the other took 2 us for 64 tokens
  uint64_t same = ~uint64_t(0);
#pragma unroll
  for (int b = 0; b < 13; ++b) {
    const bool bit = group >> b & 1;
    const uint64_t set = __ballot(bit);  // of every lane, whatever its own bit
    same &= bit ? set : ~set;
  }
  static_assert(kMaxAdapters < (1 << 13) - 1, "numbers of 13 bits");
  const int rank = __popcll(same & ((uint64_t(1) << lane) - 1));
  const bool start = group >= 0 && rank % 16 == 0;
  const uint64_t starts = __ballot(start);
  const uint32_t pieces = uint32_t(__popcll(starts)) * each.by, work = xcd_piece(at, pieces);
  if (work >= pieces) return false;
  const int item = int(each(work));
  piece = int(work - uint32_t(item) * each.by);
  const int nth = __popcll(starts & ((uint64_t(1) << lane) - 1));
  const int src = __builtin_ctzll(__ballot(start && nth == item));
  t.id = __builtin_amdgcn_readlane(group, src);
  const int first = __builtin_amdgcn_readlane(rank, src);
  const bool mine = group == t.id && rank >= first && rank < first + 16;
  t.count = __popcll(__ballot(mine));
  // each of its lanes sends its number to the lane of its place (the others to one that nobody reads)
  const int token = __builtin_amdgcn_ds_permute((mine ? rank - first : 63) * 4, lane);
  t.token[0] = __builtin_amdgcn_ds_bpermute(min(lane % 16, t.count - 1) * 4, token);
  return true;
}

// The same of any round of any call; bare: tiles of tokens without an adapter count too.
template <int SUB>
__device__ __attribute__((always_inline)) inline bool find_tile(const Adapters& l, uint32_t round, FastDiv window, FastDiv each,
                                                                bool bare, TileTokens<SUB>& t, int& piece) {
  if constexpr (SUB == 1)
    if (l.few) return few_tile(l, round, each, bare, t, piece);
  const uint32_t w = window(round), at = round - w * window.by;
  uint32_t item;
  if constexpr (SUB == 1) {
    // few tokens for each adapter, whose matrices are not met again: tiles as they come, looked up without waiting
    item = each(at);
    piece = int(at - item * each.by);
    if (item >= uint32_t(l.tile_cap)) return false;
  } else {
    // tiles without an adapter are less work: the XCDs share the others first, and then these
    const uint32_t pieces = uint32_t(gload<int32_t>(l.tile_count + 2 * w + 1)) * each.by;
    const uint32_t all = bare ? uint32_t(gload<int32_t>(l.tile_count + 2 * w)) * each.by : pieces;
    const uint32_t full = (pieces + kXcds - 1) / kXcds * kXcds;
    const uint32_t work = at < full ? xcd_piece(at, pieces) : pieces + xcd_piece(at - full, all - pieces);
    if (work >= (at < full ? pieces : all)) return false;
    item = each(work);
    piece = int(work - item * each.by);
  }
  static_assert(sizeof(AdapterTile) == 16, "one load");
  const u32x4 v = gload<u32x4>(l.tiles + int64_t(w) * l.tile_cap + item);  // id, first, count
  if (SUB == 1 && int(item) >= gload<int32_t>(l.tile_count + 2 * w + (bare ? 0 : 1))) return false;
  t.id = __builtin_amdgcn_readfirstlane(int(v[0]));
  t.count = __builtin_amdgcn_readfirstlane(int(v[2]));
#pragma unroll
  for (int m = 0; m < SUB; ++m)
    t.token[m] = gload<int32_t>(l.order + int(v[1]) + min(int(threadIdx.x & 15) + 16 * m, t.count - 1));
  return true;
}

// rounds of a product, and workgroups of its launch, which go on to further rounds if there are more
inline uint32_t adapter_rounds(const Adapters& l, FastDiv window) { return uint32_t(l.windows) * window.by; }
inline uint32_t adapter_grid(uint32_t rounds) { return std::min(rounds, uint32_t(1) << 22); }

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

// A row's last columns, fewer than eight, from column c on (none of them where
// it has ended); the loop is not unrolled, to keep the code short.
template <typename B>
__device__ __attribute__((always_inline)) inline B __attribute__((ext_vector_type(8))) last_columns(const B* row, int c, int width) {
  B __attribute__((ext_vector_type(8))) v{};
#pragma nounroll
  for (int i = width - 1; i >= c; --i) {
#pragma unroll
    for (int j = 7; j > 0; --j) v[j] = v[j - 1];
    v[0] = gload<B>(row + i);
  }
  return v;
}

// h as the matrix instructions' second operand: 16-bit parts that add up to its
// 32 bits.  bf16 takes two for a 16-bit y (which keeps 16 bits of h: 2^-18 off,
// against y's own 2^-9) and three for a 32-bit one, fp16 two (22 bits), with
// each token's row brought into fp16's range by a power of two.
template <typename E, typename Y>
constexpr int kAdapterParts = !__is_same(E, _Float16) && sizeof(Y) == 4 ? 3 : 2;

// fp16: a token's values (in four lanes, COUNT each) scaled so that the largest lies in 2^13 .. 2^14, and the factor
// that takes it back
template <int COUNT>
__device__ __attribute__((always_inline)) inline float to_half_range(float (&v)[COUNT]) {
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < COUNT; ++i) top = fmaxf(top, fabsf(v[i]));
  top = fmaxf(top, __shfl_xor(top, 16));
  top = fmaxf(top, __shfl_xor(top, 32));
  const int e = top > 0.f && top < __builtin_huge_valf() ? 14 - __builtin_amdgcn_frexp_expf(top) : 0;
#pragma unroll
  for (int i = 0; i < COUNT; ++i) v[i] = __builtin_ldexpf(v[i], e);
  return __builtin_ldexpf(1.f, -e);
}

template <typename E, int PARTS>
__device__ __attribute__((always_inline)) inline void split_parts(const float* v, u32x4 (&out)[PARTS]) {
  typedef E elem8 __attribute__((ext_vector_type(8)));
  elem8 part[PARTS];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float left = v[i];
#pragma unroll
    for (int p = 0; p < PARTS; ++p) {
      part[p][i] = E(left);
      const float is = float(part[p][i]);
      left = __builtin_isfinite(is) ? left - is : 0.f;
    }
  }
#pragma unroll
  for (int p = 0; p < PARTS; ++p) out[p] = (u32x4)part[p];
}

// Up to 16 ranks: two parts in one operand of 32, the third (with zeros behind) in a second.  q: the lane's quarter.
template <typename E, int PARTS>
__device__ __attribute__((always_inline)) inline void pack_parts(const float* v, int q, u32x4 (&out)[(PARTS + 1) / 2]) {
  u32x4 part[PARTS];
  split_parts<E, PARTS>(v, part);
  out[0] = q < 2 ? part[0] : part[1];
  if constexpr (PARTS == 3) out[1] = q < 2 ? part[2] : u32x4{};
}

}  // namespace ftmoe
