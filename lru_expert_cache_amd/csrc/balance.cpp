// C entry points of the router's balance: argument checks and the layout of the scratch memory.
#include <cmath>

#include "balance.h"
#include "entry.h"

using namespace ftmoe;

namespace {

int check_balance(const ft_moe_balance* d, ft_moe_balance& o) {
  if (!d) return bad("NULL description");
  o = *d;
  if (o.dtype < FT_DT_BF16 || o.dtype > FT_DT_F32) return bad("unknown dtype");
  if (!dim_ok(o.tokens, 0) || o.experts < 1 || o.experts > kMaxExperts || o.top_k < 1 ||
      o.top_k > std::min(o.experts, 16)) {
    set_error("bad sizes: tokens %d, experts %d (at most %d), top_k %d (at most 16 and the experts)", o.tokens,
              o.experts, kMaxExperts, o.top_k);
    return FT_E_INVALID;
  }
  if (!std::isfinite(o.weight)) return bad("weight is not finite");
  if (!row_ok(o.ld_logits, o.experts)) return bad("a row distance (ld_*) is smaller than its row, or 2^32 or more");
  return FT_OK;
}

struct BalanceWork {
  float* p;
  int32_t *c, *v, *arrived;
  double* share;
  int64_t bytes;
};
BalanceWork balance_work(const ft_moe_balance& d, void* base) {
  BalanceWork w{};
  Carve c{static_cast<uint8_t*>(base)};
  const int64_t groups = balance_groups(d.tokens);
  w.p = reinterpret_cast<float*>(c.take(groups * balance_width(d.experts) * 4));
  w.c = reinterpret_cast<int32_t*>(c.take(groups * balance_width(d.experts) * 4));
  w.v = reinterpret_cast<int32_t*>(c.take(groups * 4));
  w.share = reinterpret_cast<double*>(c.take(kMaxExperts / 16 * 8));
  w.arrived = reinterpret_cast<int32_t*>(c.take(4));
  w.bytes = c.used;
  return w;
}

}  // namespace

extern "C" {

int ft_moe_balance_work(const ft_moe_balance* desc, int64_t* bytes) {
  return guarded([&]() -> int {
    ft_moe_balance d;
    if (const int rc = check_balance(desc, d)) return rc;
    if (!bytes) return bad("bytes is NULL");
    *bytes = balance_work(d, nullptr).bytes;
    return FT_OK;
  });
}

int ft_moe_balance_forward(const ft_moe_balance* desc, const void* logits, const uint8_t* valid, int32_t* sel, float* w,
                           int32_t* counts, float* loss, void* work, int64_t work_bytes, void* hip_stream) {
  return guarded([&]() -> int {
    ft_moe_balance d;
    if (const int rc = check_balance(desc, d)) return rc;
    const BalanceWork k = balance_work(d, work);
    if (const int rc = check_work(work, work_bytes, k.bytes)) return rc;
    const int64_t es = size_of(d.dtype), T = d.tokens, E = d.experts;
    const Rows in[] = {{logits, T, E * es, d.ld_logits * es}, {valid, 1, T, 0}};
    const Rows out[] = {{sel, T ? 1 : 0, T * d.top_k * 4, 0}, {w, T ? 1 : 0, T * d.top_k * 4, 0}, {counts, 1, (E + 1) * 4, 0},
                        {loss, 1, 4, 0}, {work, 1, k.bytes, 0}};
    for (int i = 0; i < 5; ++i) {
      for (const Rows& r : in)
        if (overlap(out[i], r)) return bad("an output overlaps an input");
      for (int j = 0; j < i; ++j)
        if (overlap(out[i], out[j])) return bad("two outputs overlap");
    }
    const hipStream_t s = static_cast<hipStream_t>(hip_stream);
    DeviceGuard g;
    const Arg any{counts, 4, "counts"};
    if (const int rc = g.enter(s, {any, {loss, 4, "loss"}, {work, 16, "work"}, T ? Arg{logits, es, "logits"} : any,
                                   T && valid ? Arg{valid, 1, "valid"} : any, T ? Arg{sel, 4, "sel"} : any,
                                   T ? Arg{w, 4, "w"} : any}))
      return rc;
    BalanceForward a{};
    a.logits = logits;
    a.valid = valid;
    a.sel = sel;
    a.w = w;
    a.counts = counts;
    a.loss = loss;
    a.part_p = k.p;
    a.part_c = k.c;
    a.part_v = k.v;
    a.share = k.share;
    a.arrived = k.arrived;
    a.ld_part = balance_width(d.experts);
    a.ld = d.ld_logits;
    a.tokens = d.tokens;
    a.experts = d.experts;
    a.top_k = d.top_k;
    a.groups = balance_groups(d.tokens);
    a.weight = d.weight;
    FT_HIP_CHECK(launch_balance(d.dtype, a, s));
    return FT_OK;
  });
}

int ft_moe_balance_backward(const ft_moe_balance* desc, const void* logits, const uint8_t* valid, const int32_t* sel,
                            const float* w, const int32_t* counts, const float* dw, const float* dloss, void* dlogits,
                            void* hip_stream) {
  return guarded([&]() -> int {
    ft_moe_balance d;
    if (const int rc = check_balance(desc, d)) return rc;
    if (d.tokens == 0) return FT_OK;
    const int64_t es = size_of(d.dtype), T = d.tokens, E = d.experts, pairs = T * d.top_k * 4;
    const Rows z = {logits, T, E * es, d.ld_logits * es}, dz = {dlogits, T, E * es, d.ld_logits * es};
    const Rows in[] = {{valid, 1, T, 0}, {dw ? sel : nullptr, 1, pairs, 0}, {dw ? w : nullptr, 1, pairs, 0},
                       {counts, 1, (E + 1) * 4, 0}, {dw, 1, pairs, 0}, {dloss, 1, 4, 0}};
    if (overlap(dz, z) && !same_rows(dz, z)) return bad("dlogits overlaps logits in another way than row by row");
    for (const Rows& r : in)
      if (overlap(dz, r)) return bad("an output overlaps an input");
    const hipStream_t s = static_cast<hipStream_t>(hip_stream);
    DeviceGuard g;
    const Arg any{counts, 4, "counts"};
    if (const int rc = g.enter(s, {any, {logits, es, "logits"}, {dlogits, es, "dlogits"}, valid ? Arg{valid, 1, "valid"} : any,
                                   dw ? Arg{sel, 4, "sel"} : any, dw ? Arg{w, 4, "w"} : any,
                                   dw ? Arg{dw, 4, "dw"} : any, dloss ? Arg{dloss, 4, "dloss"} : any}))
      return rc;
    BalanceBackward a{};
    a.logits = logits;
    a.valid = valid;
    a.sel = sel;
    a.w = w;
    a.counts = counts;
    a.dw = dw;
    a.dloss = dloss;
    a.dlogits = dlogits;
    a.ld = d.ld_logits;
    a.tokens = d.tokens;
    a.experts = d.experts;
    a.top_k = d.top_k;
    a.weight = d.weight;
    FT_HIP_CHECK(launch_balance_backward(d.dtype, a, s));
    return FT_OK;
  });
}

}  // extern "C"
