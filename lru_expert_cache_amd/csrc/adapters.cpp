// C entry points of the adapters: argument checks and the layout of the scratch memory.
#include "adapters.h"
#include "entry.h"

using namespace ftmoe;

namespace {

constexpr int32_t kMaxRank = 256;

int check_adapters(const ft_moe_adapters* d, ft_moe_adapters& o) {
  if (!d) return bad("NULL description");
  o = *d;
  if (o.dtype != FT_DT_BF16 && o.dtype != FT_DT_F16) return bad("dtype must be FT_DT_BF16 or FT_DT_F16");
  if (o.out_dtype == 0) o.out_dtype = o.dtype;
  if (o.base_dtype == 0) o.base_dtype = o.out_dtype;
  if (o.out_dtype != o.dtype && o.out_dtype != FT_DT_F32) return bad("out_dtype must be dtype or FT_DT_F32");
  if (o.base_dtype != o.out_dtype && o.base_dtype != FT_DT_F32)
    return bad("base_dtype must be out_dtype or FT_DT_F32");
  if (!dim_ok(o.tokens, 0) || !dim_ok(o.in, 1) || !dim_ok(o.out, 1) || o.rank < 1 || o.rank > kMaxRank ||
      o.adapters < 1 || o.adapters > kMaxAdapters) {
    set_error("bad sizes: tokens %d, in %d, out %d, rank %d (at most %d), adapters %d (at most %d)", o.tokens, o.in,
              o.out, o.rank, kMaxRank, o.adapters, kMaxAdapters);
    return FT_E_INVALID;
  }
  if (!row_ok(o.ld_x, o.in) || !row_ok(o.ld_a, o.in) || !row_ok(o.ld_b, o.rank) || !row_ok(o.ld_base, o.out) ||
      !row_ok(o.ld_y, o.out))
    return bad("a row distance (ld_*) is smaller than its row, or 2^32 or more");
  // every byte offset within 62 bits
  if (double(o.adapters) * o.out * double(o.ld_b) * 2 > 0x1p62) return bad("the adapters' matrices take 2^62 bytes or more");
  return FT_OK;
}

struct AdaptersWork {
  AdapterPlan plan;
  float* h;
  int32_t *order, *tile_count;
  AdapterTile* tiles;
  int32_t ld_h;
  int64_t bytes;
};
AdaptersWork adapters_work(const ft_moe_adapters& d, void* base) {
  AdaptersWork w{};
  if (d.tokens == 0) return w;  // no tiles to cut
  Carve c{static_cast<uint8_t*>(base)};
  w.plan = adapter_plan(d.tokens, d.in, d.out, d.rank, d.adapters, int(size_of(d.base_dtype)), int(size_of(d.out_dtype)));
  w.ld_h = int32_t(up(d.rank, 4));
  if (w.plan.once) {  // h never leaves the workgroups: the smallest piece, so that every call with tokens has its `work`
    w.bytes = kAlign;
    return w;
  }
  w.h = reinterpret_cast<float*>(c.take(int64_t(w.plan.parts) * d.tokens * w.ld_h * 4));
  if (!w.plan.few) {
    w.order = reinterpret_cast<int32_t*>(c.take(int64_t(d.tokens) * 4));
    w.tile_count = reinterpret_cast<int32_t*>(c.take(int64_t(w.plan.windows) * 8));
    w.tiles = reinterpret_cast<AdapterTile*>(c.take(int64_t(w.plan.windows) * w.plan.tile_cap * int64_t(sizeof(AdapterTile))));
  }
  w.bytes = c.used;
  return w;
}

}  // namespace

extern "C" {

int ft_moe_adapters_work(const ft_moe_adapters* desc, int64_t* bytes) {
  return guarded([&]() -> int {
    ft_moe_adapters d;
    if (const int rc = check_adapters(desc, d)) return rc;
    if (!bytes) return bad("bytes is NULL");
    *bytes = adapters_work(d, nullptr).bytes;
    return FT_OK;
  });
}

int ft_moe_adapters_apply(const ft_moe_adapters* desc, const void* x, const int32_t* ids, const void* a, const void* b,
                          const float* scale, const void* base, void* y, void* work, int64_t work_bytes,
                          void* hip_stream) {
  return guarded([&]() -> int {
    ft_moe_adapters d;
    if (const int rc = check_adapters(desc, d)) return rc;
    if (d.tokens == 0) return FT_OK;
    const AdaptersWork w = adapters_work(d, work);
    if (const int rc = check_work(work, work_bytes, w.bytes)) return rc;
    const int64_t bs = size_of(d.base_dtype), os = size_of(d.out_dtype), T = d.tokens, n = d.adapters;
    const Rows in[] = {{base, T, d.out * bs, d.ld_base * bs}, {x, T, int64_t(d.in) * 2, d.ld_x * 2}, {ids, 1, T * 4, 0},
                       {a, n * d.rank, int64_t(d.in) * 2, d.ld_a * 2}, {b, n * d.out, int64_t(d.rank) * 2, d.ld_b * 2},
                       {scale, 1, n * 4, 0}};
    const Rows out = {y, T, d.out * os, d.ld_y * os}, scratch = {work, 1, w.bytes, 0};
    const bool in_place = same_rows(out, in[0]);
    for (int i = 0; i < 6; ++i)
      if ((overlap(out, in[i]) && !(i == 0 && in_place)) || overlap(scratch, in[i]))
        return bad("an output overlaps an input");
    if (overlap(out, scratch)) return bad("y overlaps the scratch memory");
    const hipStream_t s = static_cast<hipStream_t>(hip_stream);
    DeviceGuard g;
    if (const int rc = g.enter(s, {{x, 2, "x"}, {ids, 4, "ids"}, {a, 2, "a"}, {b, 2, "b"},
                                   {scale ? static_cast<const void*>(scale) : ids, 4, "scale"},
                                   {base ? base : y, base ? bs : os, "base"}, {y, os, "y"}, {work, 16, "work"}}))
      return rc;
    Adapters l{};
    l.x = x;
    l.ids = ids;
    l.a = a;
    l.b = b;
    l.scale = scale;
    l.base = base;
    l.y = y;
    l.h = w.h;
    l.ld_x = d.ld_x;
    l.ld_a = d.ld_a;
    l.ld_b = d.ld_b;
    l.ld_base = d.ld_base;
    l.ld_y = d.ld_y;
    l.tokens = d.tokens;
    l.in = d.in;
    l.out = d.out;
    l.rank = d.rank;
    l.count = d.adapters;
    l.in_place = in_place;
    l.order = w.order;
    l.tile_count = w.tile_count;
    l.tiles = w.tiles;
    l.ld_h = w.ld_h;
    l.few = w.plan.few;
    l.sub = w.plan.sub;
    l.windows = w.plan.windows;
    l.tile_cap = w.plan.tile_cap;
    l.parts = w.plan.parts;
    l.out_blocks = w.plan.out_blocks;
    const uint32_t rows = d.rank <= 64 ? 1 : uint32_t(d.rank + 63) / 64;  // blocks of up to 64 rows of A
    const uint32_t wide = uint32_t(w.plan.out_step) * uint32_t(l.out_blocks);
    l.by_parts = FastDiv(uint32_t(l.parts));
    l.in_each = FastDiv(rows * uint32_t(l.parts));
    l.out_each = FastDiv((uint32_t(d.out) + wide - 1) / wide);
    l.in_window = FastDiv(uint32_t(up(int64_t(l.tile_cap) * l.in_each.by, 8)));
    l.out_window = FastDiv(uint32_t(up(int64_t(l.tile_cap) * l.out_each.by, 8) + 8));  // two ranges, each a multiple
    if (w.plan.once) {
      FT_HIP_CHECK(launch_adapters_few(d.dtype, d.base_dtype, d.out_dtype, l, s));
      return FT_OK;
    }
    if (!l.few) FT_HIP_CHECK(launch_adapters_plan(l, s));
    FT_HIP_CHECK(launch_adapters_in(d.dtype, l, s));
    FT_HIP_CHECK(launch_adapters_out(d.dtype, d.base_dtype, d.out_dtype, l, s));
    return FT_OK;
  });
}

}  // extern "C"
