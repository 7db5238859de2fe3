// Low-rank adapters beside a projection: what the entry points and kernels share.
//
// Two products: h = A x and y = base + scale B h.  Tokens of the same adapter
// are brought together in tiles of 16, 32 or 64, so that its matrices are read
// once for a tile and the products run on the matrix cores; a token's own
// result does not depend on which others share its tile.  h goes through
// memory in 32 bits: the first product is cut along K over as many workgroups
// as fill the card, and the second adds their parts, in order.  Few tokens of
// narrow projections have both in one launch, where every workgroup forms h
// for itself.
#pragma once
#include "common.h"
#include "gmem.h"

namespace ftmoe {

constexpr int32_t kMaxAdapters = 4096;  // counters of the grouping, in LDS
// Tokens are grouped within windows of this many.
constexpr int32_t kAdapterWindow = 8192;
// Up to this many, each wave finds its tile by itself; else a launch of its own writes down the tiles.
constexpr int32_t kAdapterFew = 64;

// Division of a number below 2^31 by one that is known before the launch.
struct FastDiv {
  uint32_t by, mul, shift;
  FastDiv() = default;
  explicit FastDiv(uint32_t d) : by(d), mul(0), shift(0) {
    if (d <= 1) return;
    uint32_t bits = 1;  // 2^bits >= d
    while ((uint64_t(1) << bits) < d) ++bits;
    shift = bits - 1;
    mul = uint32_t(((uint64_t(1) << (31 + bits)) + d - 1) / d);
  }
#ifdef __HIPCC__
  __device__ __attribute__((always_inline)) inline uint32_t operator()(uint32_t n) const {
    return by <= 1 ? n : __umulhi(n, mul) >> shift;
  }
#endif
};

struct AdapterTile {
  int32_t id;     // adapter, or their number for tokens that have none
  int32_t first;  // in `order`
  int32_t count;
  int32_t unused;
};

struct Adapters {
  const void* x;
  const int32_t* ids;
  const void *a, *b;
  const float* scale;  // null: 1
  const void* base;    // null: 0
  void* y;
  float* h;            // [parts][T][ld_h]: sums over each part of K
  int32_t* order;      // [T]: tokens of each tile next to each other
  AdapterTile* tiles;  // [windows][tile_cap]
  int32_t* tile_count; // [windows][2]: all tiles, and those of an adapter, which come first
  int64_t ld_x, ld_a, ld_b, ld_base, ld_y;
  int32_t tokens, in, out, rank, count, ld_h;
  int32_t few, sub;    // tiles found by each wave; groups of 16 tokens in a tile
  int32_t windows, tile_cap, parts;
  int32_t out_blocks;  // steps of columns of y that a workgroup of the second product takes
  // either product: a tile's pieces of work, and a window's (of as many tiles as it can have; a multiple of the XCDs)
  FastDiv in_each, in_window, out_each, out_window;
  FastDiv by_parts;
  bool in_place;       // y is base: tokens without an adapter are left out
};

// Blocks of 32 columns that a wave of the second product takes at once: 128
// bytes of a row of base and y, whose halves would else be asked for by two
// waves (adapters of rank 64, 8192 tokens: half as many requests to the L2
// cache); one where two would take too many registers, and for tiles of 16
// tokens and up to 16 ranks, whose many workgroups wait for ids, h and base in
// turn: four waves a SIMD instead of three (1531 tokens, 2048 into 5000, rank
// 8, bf16: 22.2 us against 23.2, with a 32-bit base 23.3 against 25.7).
constexpr int adapter_out_blocks(int base_bytes, int out_bytes, int sub, int rank) {
  return out_bytes == 4 || (base_bytes == 4 && sub == 4) || rank > 64 || (sub == 1 && rank <= 16) ? 1 : 2;
}
// How a call of one token or more is cut: a rule on sizes and types alone.
struct AdapterPlan {
  int32_t few, sub, windows, tile_cap, parts, out_blocks;
  int32_t once;      // both products in one launch: few tokens, up to 16 ranks
  int32_t out_step;  // columns of y in a step of a workgroup: its waves' blocks
};
AdapterPlan adapter_plan(int32_t tokens, int32_t in, int32_t out, int32_t rank, int32_t count, int base_bytes,
                         int out_bytes);

hipError_t launch_adapters_plan(const Adapters& l, hipStream_t s);
hipError_t launch_adapters_in(int dtype, const Adapters& l, hipStream_t s);
hipError_t launch_adapters_few(int dtype, int base_dtype, int out_dtype, const Adapters& l, hipStream_t s);
hipError_t launch_adapters_out(int dtype, int base_dtype, int out_dtype, const Adapters& l, hipStream_t s);

}  // namespace ftmoe
