// C entry points of the root-mean-square norm: argument checks and the layout of the scratch memory.
#include <cmath>

#include "entry.h"
#include "norm.h"

using namespace ftmoe;

namespace {

int check_norm(const ft_moe_rms_norm* d, ft_moe_rms_norm& o) {
  if (!d) return bad("NULL description");
  o = *d;
  if (o.dtype < FT_DT_BF16 || o.dtype > FT_DT_F32) return bad("unknown dtype");
  if (o.residual_dtype == 0) o.residual_dtype = o.dtype;
  if (o.residual_dtype != o.dtype && o.residual_dtype != FT_DT_F32)
    return bad("residual_dtype must be dtype or FT_DT_F32");
  if (!dim_ok(o.rows, 0) || !dim_ok(o.cols, 1)) {
    set_error("bad sizes: rows %d, cols %d", o.rows, o.cols);
    return FT_E_INVALID;
  }
  if (!(o.eps >= 0.f) || !std::isfinite(o.eps)) return bad("eps must be a number of 0 or more");
  if (!row_ok(o.ld_x, o.cols) || !row_ok(o.ld_residual, o.cols) || !row_ok(o.ld_sum, o.cols) ||
      !row_ok(o.ld_y, o.cols) || !row_ok(o.ld_codes, o.cols))
    return bad("a row distance (ld_*) is smaller than its row, or 2^32 or more");
  return FT_OK;
}

Rows rows_of(const ft_moe_rms_norm& d, const void* p, int64_t ld, int64_t es) {
  return {p, d.rows, d.cols * es, ld * es};
}

// one launch, whose only group of rows writes the weight's gradient itself
bool norm_once(const ft_moe_rms_norm& d) { return d.rows <= kNormOnce && norm_rows(d.cols); }

struct NormWork {
  float *stats, *part;
  int64_t bytes;
};
// what a call with or without dweight uses
NormWork norm_work(const ft_moe_rms_norm& d, bool dweight, void* base) {
  NormWork w{};
  Carve c{static_cast<uint8_t*>(base)};
  if (!norm_rows(d.cols)) w.stats = reinterpret_cast<float*>(c.take(int64_t(d.rows) * 16));
  if (dweight && !norm_once(d))
    w.part = reinterpret_cast<float*>(c.take(norm_groups(d.rows, d.cols) * norm_part_ld(d.cols) * 4));
  w.bytes = d.rows ? c.used : 0;
  return w;
}

}  // namespace

extern "C" {

int ft_moe_rms_norm_forward(const ft_moe_rms_norm* desc, const void* x, const void* residual, const void* weight,
                            void* sum, void* y, int8_t* codes, float* scale, void* hip_stream) {
  return guarded([&]() -> int {
    ft_moe_rms_norm d;
    if (const int rc = check_norm(desc, d)) return rc;
    if (d.rows == 0) return FT_OK;
    if (!codes != !scale) return bad("codes and scale are given together or not at all");
    if (!sum && !y && !codes) return FT_OK;
    const int64_t es = size_of(d.dtype), rs = size_of(d.residual_dtype);
    const Rows in[] = {rows_of(d, x, d.ld_x, es), rows_of(d, residual, d.ld_residual, rs), {weight, 1, d.cols * es, 0}};
    const Rows out[] = {rows_of(d, sum, d.ld_sum, rs), rows_of(d, y, d.ld_y, es), rows_of(d, codes, d.ld_codes, 1),
                        {scale, 1, int64_t(d.rows) * 4, 0}};
    for (int i = 0; i < 4; ++i) {
      for (int j = 0; j < 3; ++j)
        if (overlap(out[i], in[j]) && !(i < 2 && j < 2 && same_rows(out[i], in[j])))
          return bad("an output overlaps an input in another way than row by row");
      for (int j = 0; j < i; ++j)
        if (overlap(out[i], out[j])) return bad("two outputs overlap");
    }
    const hipStream_t s = static_cast<hipStream_t>(hip_stream);
    DeviceGuard g;
    if (const int rc = g.enter(s, {{x, es, "x"}, {residual ? residual : x, residual ? rs : es, "residual"},
                                   {weight, es, "weight"}, {sum ? sum : x, sum ? rs : es, "sum"}, {y ? y : x, es, "y"},
                                   {codes ? codes : x, 1, "codes"}, {scale ? scale : x, scale ? 4 : es, "scale"}}))
      return rc;
    NormForward a{};
    a.x = x;
    a.residual = residual;
    a.weight = weight;
    a.sum = sum;
    a.y = y;
    a.codes = codes;
    a.scale = scale;
    a.ld_x = d.ld_x;
    a.ld_residual = d.ld_residual;
    a.ld_sum = d.ld_sum;
    a.ld_y = d.ld_y;
    a.ld_codes = d.ld_codes;
    a.rows = d.rows;
    a.cols = d.cols;
    a.eps = d.eps;
    FT_HIP_CHECK(launch_norm(d.dtype, d.residual_dtype, a, s));
    return FT_OK;
  });
}

int ft_moe_rms_norm_work(const ft_moe_rms_norm* desc, int64_t* bytes) {
  return guarded([&]() -> int {
    ft_moe_rms_norm d;
    if (const int rc = check_norm(desc, d)) return rc;
    if (!bytes) return bad("bytes is NULL");
    *bytes = norm_work(d, true, nullptr).bytes;
    return FT_OK;
  });
}

int ft_moe_rms_norm_backward(const ft_moe_rms_norm* desc, const void* sum, const void* weight, const void* dy,
                             const void* dsum, void* dx, void* dresidual, void* dweight, void* work, int64_t work_bytes,
                             void* hip_stream) {
  return guarded([&]() -> int {
    ft_moe_rms_norm d;
    if (const int rc = check_norm(desc, d)) return rc;
    if (!dweight && (d.rows == 0 || (!dx && !dresidual))) return FT_OK;
    const NormWork w = norm_work(d, dweight != nullptr, work);
    if (const int rc = check_work(work, work_bytes, w.bytes)) return rc;
    const int64_t es = size_of(d.dtype), rs = size_of(d.residual_dtype);
    const Rows in[] = {rows_of(d, sum, d.ld_sum, rs), rows_of(d, dy, d.ld_y, es), rows_of(d, dsum, d.ld_residual, rs),
                       {weight, 1, d.cols * es, 0}};
    const Rows out[] = {rows_of(d, dx, d.ld_x, es), rows_of(d, dresidual, d.ld_residual, rs),
                        {dweight, 1, d.cols * es, 0}, {w.bytes ? work : nullptr, 1, w.bytes, 0}};
    for (int i = 0; i < 4; ++i) {
      for (int j = 0; j < 4; ++j)
        if (overlap(out[i], in[j]) && !(i < 2 && j < 3 && same_rows(out[i], in[j])))
          return bad("an output overlaps an input in another way than row by row");
      for (int j = 0; j < i; ++j)
        if (overlap(out[i], out[j])) return bad("two outputs overlap");
    }
    const hipStream_t s = static_cast<hipStream_t>(hip_stream);
    const bool some = d.rows > 0;
    const void* any = dweight ? dweight : dx ? dx : dresidual;
    const int64_t as = dweight || dx ? es : rs;
    auto arg = [&](bool read, const void* p, int64_t align, const char* name) {
      return read ? Arg{p, align, name} : Arg{any, as, name};
    };
    DeviceGuard g;
    if (const int rc = g.enter(s, {arg(some, sum, rs, "sum"), arg(some, weight, es, "weight"), arg(some, dy, es, "dy"),
                                   arg(some && dsum, dsum, rs, "dsum"), arg(some && dx, dx, es, "dx"),
                                   arg(some && dresidual, dresidual, rs, "dresidual"),
                                   arg(dweight != nullptr, dweight, es, "dweight"),
                                   arg(w.bytes > 0, work, 16, "work")}))
      return rc;
    NormBackward a{};
    a.sum = sum;
    a.weight = weight;
    a.dy = dy;
    a.dsum = dsum;
    a.dx = dx;
    a.dresidual = dresidual;
    const bool once = some && dweight && norm_once(d);
    a.dweight = once ? dweight : nullptr;
    a.part = w.part;
    a.stats = w.stats;
    a.ld_sum = d.ld_sum;
    a.ld_y = d.ld_y;
    a.ld_residual = d.ld_residual;
    a.ld_x = d.ld_x;
    a.rows = d.rows;
    a.cols = d.cols;
    a.groups = once ? 1 : norm_groups(d.rows, d.cols);
    a.eps = d.eps;
    if (some) FT_HIP_CHECK(launch_norm_backward(d.dtype, d.residual_dtype, a, s));
    if (dweight && !once) FT_HIP_CHECK(launch_norm_join(d.dtype, w.part, a.groups, d.cols, dweight, s));
    return FT_OK;
  });
}

}  // extern "C"
