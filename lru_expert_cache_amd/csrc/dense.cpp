// C entry points of the dense feed-forward operators: argument checks, the
// layout of the scratch memory, and the sequence of products of each call.
#include "dense.h"
#include "entry.h"

using namespace ftmoe;

namespace {

constexpr int32_t kMaxIntK = 131071;  // 128 * 128 * K < 2^31

// checks a block's description and fills in the row distances
int check_ffn(const ft_moe_gated_ffn* d, ft_moe_gated_ffn& o) {
  if (!d) return bad("NULL description");
  o = *d;
  if (o.dtype != FT_DT_BF16 && o.dtype != FT_DT_F16) return bad("dtype must be FT_DT_BF16 or FT_DT_F16");
  if (!dim_ok(o.tokens, 0) || !dim_ok(o.hidden, 1) || !dim_ok(o.inter, 1)) {
    set_error("bad sizes: tokens %d, hidden %d, inter %d", o.tokens, o.hidden, o.inter);
    return FT_E_INVALID;
  }
  if (!row_ok(o.ld_x, o.hidden) || !row_ok(o.ld_y, o.hidden) || !row_ok(o.ld_gu, 2 * int64_t(o.inter)) ||
      !row_ok(o.ld_w_in, o.hidden) || !row_ok(o.ld_w_out, o.inter))
    return bad("a row distance (ld_*) is smaller than its row, or 2^32 or more");
  return FT_OK;
}

const uint8_t* u8(const void* p) { return static_cast<const uint8_t*>(p); }
uint8_t* u8(void* p) { return static_cast<uint8_t*>(p); }

DenseProblem product(const void* a, int64_t lda, const void* b, int64_t ldb, int m, int n, int k, void* c, int64_t ldc,
                     int64_t es) {
  DenseProblem p{};
  p.a[0] = p.a[1] = u8(a);
  p.b[0] = p.b[1] = u8(b);
  p.lda = lda * es;
  p.ldb = ldb * es;
  p.m = m;
  p.n = n;
  p.k = k;
  p.segs = 1;
  p.c = u8(c);
  p.ldc = ldc;
  return p;
}

DenseShape shape(const DenseProblem& p) { return {p.m, p.n, p.k, p.segs}; }

// products that dense_few.hip runs
bool dense_few(DenseForm form, const DenseShape* shapes, int count) {
  return dense_a_rows(form) && dense_b_rows(form) && count == 1 && shapes[0].m <= kDenseFewRows;
}

// scratch bytes for the parts of a product's K
int64_t parts_bytes(DenseForm form, std::initializer_list<DenseShape> shapes) {
  if (dense_few(form, shapes.begin(), int(shapes.size()))) return 0;
  const int splits = dense_plan(form, shapes.begin(), int(shapes.size())).splits;
  int64_t n = 0;
  for (const DenseShape& s : shapes) n += up(dense_part_bytes(form, s, splits), kAlign);
  return n;
}

// One launch (two when K is cut into parts): up to three products of one form.
// clear: queue counters that a tiled launch sets to zero.
int run(DenseForm form, int dtype, std::initializer_list<DenseProblem> problems, uint8_t* part, hipStream_t s,
        uint32_t* clear = nullptr) {
  DenseLaunch l{};
  DenseShape shapes[kDenseMaxProblems];
  bool tiled = true;
  for (const DenseProblem& p : problems) {
    tiled = tiled && dense_tileable(form, p);
    shapes[l.count] = shape(p);
    l.p[l.count++] = p;
  }
  l.splits = 1;
  if (!tiled) {
    FT_HIP_CHECK(launch_dense_any(form, dtype, l, s));
    return FT_OK;
  }
  if (dense_few(form, shapes, l.count)) {
    FT_HIP_CHECK(launch_dense_few(form, dtype, l, s));
    return FT_OK;
  }
  const DensePlan plan = dense_plan(form, shapes, l.count);
  l.splits = plan.splits;
  l.clear = clear;
  for (int i = 0; i < l.count && plan.splits > 1; ++i) {
    l.p[i].part = part;
    part += up(dense_part_bytes(form, shapes[i], plan.splits), kAlign);
  }
  FT_HIP_CHECK(launch_dense_tile(form, dtype, plan.tile, l, s));
  return FT_OK;
}

// An 8-bit product whose tokens lie at x (ld_x elements of type dtype apart)
// and are quantised to p's a and xs: by the product itself where it can, in a
// launch of its own otherwise.
int run_quantized(DenseForm form, int out_dtype, DenseProblem p, int dtype, const void* x, int64_t ld_x, uint8_t* part,
                  hipStream_t s) {
  if (dense_few_quantizes(p.m, p.k) && dense_tileable(form, p)) {
    p.a[0] = p.a[1] = u8(x);
    p.lda = ld_x * (dtype == FT_DT_F32 ? 4 : 2);
    p.tokens = dtype;
    DenseLaunch l{};
    l.p[0] = p;
    l.count = l.splits = 1;
    FT_HIP_CHECK(launch_dense_few(form, out_dtype, l, s));
    return FT_OK;
  }
  FT_HIP_CHECK(launch_int_quantize(dtype, p.m, p.k, x, ld_x, const_cast<int8_t*>(reinterpret_cast<const int8_t*>(p.a[0])),
                                   p.lda, const_cast<float*>(p.xs), s));
  return run(form, out_dtype, {p}, part, s);
}

// A call's operands that the tiled kernels cannot take as they lie, copied into
// scratch memory.  Whether one is copied depends on sizes and row distances
// only (the scratch memory is sized before addresses are known); a base
// address off the 16-byte grid leaves its product to the general kernel.
struct Packs {
  DensePackLaunch l{};
  Carve* c;
  bool odd(int64_t width, int64_t ld, int64_t es) const { return width * es % 16 || ld * es % 16; }
  // a matrix: where it then lies, and its rows' distance; one that the call does not read keeps its place only
  const void* matrix(const void* src, int64_t rows, int64_t width, int64_t& ld, int64_t es, bool& whole, bool read = true) {
    whole = false;
    if (!odd(width, ld, es)) return src;
    const int64_t to = up(width * es, 128);
    uint8_t* dst = c->take(rows * to);
    add({u8(src), dst, ld * es, to, width * es, to, read ? rows : 0});
    ld = to / es;
    whole = true;
    return dst;
  }
  // zeros behind the rows of a matrix of the call's own, up to a whole piece; whether there are any.  The piece that
  // the rows end in is cleared before its values are written.
  bool behind(uint8_t* base, int64_t rows, int64_t width, int64_t ld, int64_t es) {
    if (width * es % 16 == 0) return false;
    const int64_t from = width * es / 16 * 16;
    add({nullptr, base + from, 0, ld * es, 0, 16, rows});
    return true;
  }
  void add(const DensePack& p) { l.p[l.count++] = p; }
};

// ------------------------------------------------------------ gated block
struct FfnWork {
  int64_t ldi;  // elements between rows of h, and half of a row of dgu
  uint8_t *h, *dgu, *part;
  int32_t lo;   // rows from an h, dg or du to what its rounding left off, 0 with more than a few tokens
  int64_t rows; // of h and dgu
  uint32_t* queue;
  // the operands as the products take them
  const void *x, *dy, *wg, *wu, *wd;
  int64_t ld_x, ld_y, ld_in, ld_out;
  bool whole_x, whole_y, whole_in, whole_out, whole_i;
  DensePackLaunch packs;
  int64_t bytes;
};
// read_x, read_in: whether the call reads x, and w_gate and w_up
FfnWork ffn_work(const ft_moe_gated_ffn& d, bool backward, void* base, const void* x = nullptr, const void* dy = nullptr,
                 const void* wg = nullptr, const void* wu = nullptr, const void* wd = nullptr, bool read_x = true,
                 bool read_in = true) {
  FfnWork w{};
  Carve c{static_cast<uint8_t*>(base)};
  const int T = d.tokens, H = d.hidden, I = d.inter;
  w.ldi = up(I, 64);
  w.lo = dense_lo(T, backward);
  w.rows = int64_t(T) + w.lo;
  w.h = c.take(w.rows * w.ldi * 2);
  int64_t part;
  if (backward) {
    w.dgu = c.take(w.rows * w.ldi * 4);
    w.queue = reinterpret_cast<uint32_t*>(c.take(kDenseQueue * 4));
    const int segs = w.lo ? 2 : 1;
    part = std::max({parts_bytes(kDenseGrad, {{T, I, H, 1}}), parts_bytes(kDenseCols, {{T, H, I, 2}}),
                     parts_bytes(kDenseOuter, {{I, H, T, segs}, {I, H, T, segs}, {H, I, T, segs}})});
  } else {
    part = std::max(parts_bytes(kDenseGated, {{T, I, H, 1}}), parts_bytes(kDenseRows, {{T, H, I, 1}}));
  }
  w.part = c.take(part);
  Packs k;
  k.c = &c;
  w.ld_x = d.ld_x;
  w.ld_y = d.ld_y;
  w.ld_in = d.ld_w_in;
  w.ld_out = d.ld_w_out;
  if (T > 0) {
    int64_t ld_up = d.ld_w_in;
    w.x = k.matrix(x, T, H, w.ld_x, 2, w.whole_x, read_x);
    w.wg = k.matrix(wg, I, H, w.ld_in, 2, w.whole_in, read_in);
    w.wu = k.matrix(wu, I, H, ld_up, 2, w.whole_in, read_in);
    w.wd = k.matrix(wd, H, I, w.ld_out, 2, w.whole_out);
    if (backward) w.dy = k.matrix(dy, T, H, w.ld_y, 2, w.whole_y);
    w.whole_i = k.behind(w.h, w.rows, I, w.ldi, 2);
    if (backward) {
      k.behind(w.dgu, w.rows, I, 2 * w.ldi, 2);
      k.behind(w.dgu + 2 * w.ldi, w.rows, I, 2 * w.ldi, 2);
    }
  }
  w.packs = k.l;
  w.bytes = c.used;
  return w;
}

// ------------------------------------------------------------ 8-bit
int check_product(const ft_moe_int_product* d, ft_moe_int_product& o) {
  if (!d) return bad("NULL description");
  o = *d;
  if (o.out_dtype < FT_DT_BF16 || o.out_dtype > FT_DT_F32) return bad("unknown out_dtype");
  if (!dim_ok(o.tokens, 0) || !dim_ok(o.out, 1) || o.in < 1 || o.in > kMaxIntK) {
    set_error("bad sizes: tokens %d, in %d (at most %d), out %d", o.tokens, o.in, kMaxIntK, o.out);
    return FT_E_INVALID;
  }
  if (!row_ok(o.ld_x, o.in) || !row_ok(o.ld_w, o.in) || !row_ok(o.ld_y, o.out))
    return bad("a row distance (ld_*) is smaller than its row, or 2^32 or more");
  return FT_OK;
}
struct IntWork {
  int64_t ldx, ldh, ldf;
  int8_t *xq, *hq;
  float *xs, *hs, *h;
  uint8_t* part;
  const void *wg, *wu, *wd;
  int64_t ld_in, ld_out;
  bool whole_x, whole_h, whole_in, whole_out;
  DensePackLaunch packs;
  int64_t bytes;
};
IntWork int_work(const ft_moe_gated_ffn& d, void* base, const void* wg = nullptr, const void* wu = nullptr,
                 const void* wd = nullptr) {
  IntWork w{};
  Carve c{static_cast<uint8_t*>(base)};
  const int64_t T = d.tokens, H = d.hidden, I = d.inter;
  w.ldx = up(H, 128);
  w.ldh = up(I, 128);
  w.ldf = up(I, 32);
  w.xq = reinterpret_cast<int8_t*>(c.take(T * w.ldx));
  w.xs = reinterpret_cast<float*>(c.take(T * 4));
  w.h = reinterpret_cast<float*>(c.take(T * w.ldf * 4));
  w.hq = reinterpret_cast<int8_t*>(c.take(T * w.ldh));
  w.hs = reinterpret_cast<float*>(c.take(T * 4));
  w.part = c.take(std::max(parts_bytes(kDenseIntGated, {{d.tokens, d.inter, d.hidden, 1}}),
                           parts_bytes(kDenseInt, {{d.tokens, d.hidden, d.inter, 1}})));
  Packs k;
  k.c = &c;
  w.ld_in = d.ld_w_in;
  w.ld_out = d.ld_w_out;
  if (T > 0) {
    int64_t ld_up = d.ld_w_in;
    w.wg = k.matrix(wg, I, H, w.ld_in, 1, w.whole_in);
    w.wu = k.matrix(wu, I, H, ld_up, 1, w.whole_in);
    w.wd = k.matrix(wd, H, I, w.ld_out, 1, w.whole_out);
    w.whole_x = k.behind(reinterpret_cast<uint8_t*>(w.xq), T, H, w.ldx, 1);
    w.whole_h = k.behind(reinterpret_cast<uint8_t*>(w.hq), T, I, w.ldh, 1);
  }
  w.packs = k.l;
  w.bytes = c.used;
  return w;
}
// the product alone: its operands as it takes them
struct ProductWork {
  const void *x, *w;
  int64_t ld_x, ld_w;
  bool whole_x, whole_w;
  uint8_t* part;
  DensePackLaunch packs;
  int64_t bytes;
};
ProductWork product_work(const ft_moe_int_product& d, void* base, const void* x = nullptr, const void* wt = nullptr) {
  ProductWork w{};
  Carve c{static_cast<uint8_t*>(base)};
  w.part = c.take(parts_bytes(kDenseInt, {{d.tokens, d.out, d.in, 1}}));
  Packs k;
  k.c = &c;
  w.ld_x = d.ld_x;
  w.ld_w = d.ld_w;
  if (d.tokens > 0) {
    w.x = k.matrix(x, d.tokens, d.in, w.ld_x, 1, w.whole_x);
    w.w = k.matrix(wt, d.out, d.in, w.ld_w, 1, w.whole_w);
  }
  w.packs = k.l;
  w.bytes = c.used;
  return w;
}
int check_int_ffn(const ft_moe_gated_ffn* d, ft_moe_gated_ffn& o) {
  if (const int rc = check_ffn(d, o)) return rc;
  if (o.hidden > kMaxIntK || o.inter > kMaxIntK) {
    set_error("bad sizes: hidden %d, inter %d (8 bit: at most %d)", o.hidden, o.inter, kMaxIntK);
    return FT_E_INVALID;
  }
  return FT_OK;
}

}  // namespace

extern "C" {

int ft_moe_gated_ffn_work(const ft_moe_gated_ffn* d, int32_t backward, int64_t* bytes) {
  return guarded([&]() -> int {
    ft_moe_gated_ffn o;
    if (const int rc = check_ffn(d, o)) return rc;
    if (!bytes) return bad("bytes is NULL");
    *bytes = ffn_work(o, backward != 0, nullptr).bytes;
    return FT_OK;
  });
}

int ft_moe_gated_ffn_forward(const ft_moe_gated_ffn* desc, const void* x, const void* w_gate, const void* w_up,
                             const void* w_down, void* y, void* gu, void* work, int64_t work_bytes, void* hip_stream) {
  return guarded([&]() -> int {
    ft_moe_gated_ffn d;
    if (const int rc = check_ffn(desc, d)) return rc;
    if (d.tokens == 0) return FT_OK;
    const FfnWork w = ffn_work(d, false, work, x, nullptr, w_gate, w_up, w_down);
    if (const int rc = check_work(work, work_bytes, w.bytes)) return rc;
    if (same(y, {x, w_gate, w_up, w_down, gu, work}) || same(gu, {x, w_gate, w_up, w_down, work}) ||
        same(work, {x, w_gate, w_up, w_down}))
      return bad("an output is also another argument");
    const hipStream_t s = static_cast<hipStream_t>(hip_stream);
    DeviceGuard g;
    if (const int rc = g.enter(s, {{x, 2, "x"}, {w_gate, 2, "w_gate"}, {w_up, 2, "w_up"}, {w_down, 2, "w_down"},
                                   {y, 2, "y"}, {gu ? gu : y, 2, "gu"}, {work, 16, "work"}}))
      return rc;

    FT_HIP_CHECK(launch_dense_pack(w.packs, s));
    DenseProblem p = product(w.x, w.ld_x, w.wg, w.ld_in, d.tokens, d.inter, d.hidden, w.h, w.ldi, 2);
    p.b[1] = u8(w.wu);
    p.a_whole = w.whole_x;
    p.b_whole = w.whole_in;
    p.gu = u8(gu);
    p.ldgu = d.ld_gu;
    p.off_u = d.inter;
    p.c_lo = w.lo;
    if (const int rc = run(kDenseGated, d.dtype, {p}, w.part, s)) return rc;
    p = product(w.h, w.ldi, w.wd, w.ld_out, d.tokens, d.hidden, d.inter, y, d.ld_y, 2);
    p.a_lo = w.lo;
    p.a_whole = w.whole_i;
    p.b_whole = w.whole_out;
    return run(kDenseRows, d.dtype, {p}, w.part, s);
  });
}

int ft_moe_gated_ffn_backward(const ft_moe_gated_ffn* desc, const void* x, const void* w_gate, const void* w_up,
                              const void* w_down, const void* gu, const void* dy, void* dx, void* dw_gate, void* dw_up,
                              void* dw_down, void* work, int64_t work_bytes, void* hip_stream) {
  return guarded([&]() -> int {
    ft_moe_gated_ffn d;
    if (const int rc = check_ffn(desc, d)) return rc;
    const bool grads = dw_gate || dw_up || dw_down;
    if (grads && !(dw_gate && dw_up && dw_down)) return bad("weight gradients are given together or not at all");
    if (!grads && (!dx || d.tokens == 0)) return FT_OK;
    const FfnWork w = ffn_work(d, true, work, x, dy, w_gate, w_up, w_down, grads, dx != nullptr);
    if (const int rc = check_work(work, work_bytes, w.bytes)) return rc;
    for (const void* o : {(const void*)dx, (const void*)dw_gate, (const void*)dw_up, (const void*)dw_down, (const void*)work})
      if (same(o, {x, w_gate, w_up, w_down, gu, dy})) return bad("an output is also another argument");
    if (same(dx, {dw_gate, dw_up, dw_down, work}) || same(dw_gate, {dw_up, dw_down, work}) ||
        same(dw_up, {dw_down, work}) || same(dw_down, {work}))
      return bad("an output is given twice");
    const hipStream_t s = static_cast<hipStream_t>(hip_stream);
    const int T = d.tokens, H = d.hidden, I = d.inter;
    // what is read and written of the tokens, the weights and their gradients
    const void* any = grads ? dw_gate : dx;
    DeviceGuard g;
    if (const int rc = g.enter(s, {{T && grads ? x : any, 2, "x"}, {T && dx ? w_gate : any, 2, "w_gate"},
                                   {T && dx ? w_up : any, 2, "w_up"}, {T ? w_down : any, 2, "w_down"},
                                   {T ? gu : any, 2, "gu"}, {T ? dy : any, 2, "dy"}, {T && dx ? dx : any, 2, "dx"},
                                   {grads ? dw_gate : any, 2, "dw_gate"}, {grads ? dw_up : any, 2, "dw_up"},
                                   {grads ? dw_down : any, 2, "dw_down"}, {T ? work : any, T ? 16 : 2, "work"}}))
      return rc;

    DenseProblem cols{};
    DenseProblem outer[3];
    if (dx) {
      cols = product(w.dgu, 2 * w.ldi, w.wg, w.ld_in, T, H, I, dx, d.ld_x, 2);
      cols.a[1] = w.dgu + 2 * w.ldi;
      cols.b[1] = u8(w.wu);
      cols.segs = 2;
      cols.a_lo = w.lo;
      cols.a_whole = w.whole_i;
      cols.b_whole = w.whole_in;
    }
    if (grads) {
      outer[0] = product(w.dgu, 2 * w.ldi, w.x, w.ld_x, I, H, T, dw_gate, d.ld_w_in, 2);
      outer[1] = product(w.dgu + 2 * w.ldi, 2 * w.ldi, w.x, w.ld_x, I, H, T, dw_up, d.ld_w_in, 2);
      outer[2] = product(w.dy, w.ld_y, w.h, w.ldi, H, I, T, dw_down, d.ld_w_out, 2);
      outer[0].a_whole = outer[1].a_whole = outer[2].b_whole = w.whole_i;
      outer[0].b_whole = outer[1].b_whole = w.whole_x;
      outer[2].a_whole = w.whole_y;
      if (w.lo) {  // what the rounding left off: a second K segment
        outer[0].segs = outer[1].segs = outer[2].segs = 2;
        outer[0].a[1] = outer[0].a[0] + w.lo * outer[0].lda;
        outer[1].a[1] = outer[1].a[0] + w.lo * outer[1].lda;
        outer[2].b[1] = outer[2].b[0] + w.lo * outer[2].ldb;
      }
    }
    if (T > 0) {
      FT_HIP_CHECK(launch_dense_pack(w.packs, s));
      DenseProblem p = product(w.dy, w.ld_y, w.wd, w.ld_out, T, I, H, grads ? w.h : nullptr, w.ldi, 2);
      p.a_whole = w.whole_y;
      p.b_whole = w.whole_out;
      p.gu = const_cast<uint8_t*>(u8(gu));
      p.ldgu = d.ld_gu;
      p.off_u = I;
      p.dgu = w.dgu;
      p.lddgu = 2 * w.ldi;
      p.off_du = w.ldi;
      p.c_lo = w.lo;
      // dx and the weight gradients in one launch, where all can be tiled
      int pair = 0;
      if (dx && grads && dense_tileable(kDenseGrad, p) && dense_tileable(kDenseCols, cols) &&
          dense_tileable(kDenseOuter, outer[0]) && dense_tileable(kDenseOuter, outer[1]) &&
          dense_tileable(kDenseOuter, outer[2]))
        pair = dense_plan_pair({shape(outer[0]), shape(outer[1]), shape(outer[2])}, shape(cols), w.lo != 0);
      if (const int rc = run(kDenseGrad, d.dtype, {p}, w.part, s, pair ? w.queue : nullptr)) return rc;
      if (pair) {
        DensePair l{};
        for (int i = 0; i < 3; ++i) l.outer.p[i] = outer[i];
        l.outer.count = 3;
        l.cols.p[0] = cols;
        l.cols.count = 1;
        l.outer.splits = l.cols.splits = 1;
        l.queue = w.queue;
        FT_HIP_CHECK(launch_dense_pair(d.dtype, pair, l, s));
        return FT_OK;
      }
    }
    if (T > 0 && dx)
      if (const int rc = run(kDenseCols, d.dtype, {cols}, w.part, s)) return rc;
    if (!grads) return FT_OK;
    return run(kDenseOuter, d.dtype, {outer[0], outer[1], outer[2]}, w.part, s);
  });
}

int ft_moe_int_quantize(int32_t dtype, int32_t rows, int32_t cols, const void* x, int64_t ld_x, int8_t* codes,
                        int64_t ld_codes, float* scale, void* hip_stream) {
  return guarded([&]() -> int {
    if (dtype < FT_DT_BF16 || dtype > FT_DT_F32) return bad("unknown dtype");
    if (!dim_ok(rows, 0) || !dim_ok(cols, 1)) {
      set_error("bad sizes: rows %d, cols %d", rows, cols);
      return FT_E_INVALID;
    }
    if (!row_ok(ld_x, cols) || !row_ok(ld_codes, cols))
      return bad("a row distance (ld_*) is smaller than its row, or 2^32 or more");
    if (rows == 0) return FT_OK;
    if (same(codes, {x, scale}) || same(scale, {x})) return bad("an output is also another argument");
    const hipStream_t s = static_cast<hipStream_t>(hip_stream);
    DeviceGuard g;
    if (const int rc = g.enter(s, {{x, size_of(dtype), "x"}, {codes, 1, "codes"}, {scale, 4, "scale"}})) return rc;
    FT_HIP_CHECK(launch_int_quantize(dtype, rows, cols, x, ld_x, codes, ld_codes, scale, s));
    return FT_OK;
  });
}

int ft_moe_int_matmul_work(const ft_moe_int_product* d, int64_t* bytes) {
  return guarded([&]() -> int {
    ft_moe_int_product o;
    if (const int rc = check_product(d, o)) return rc;
    if (!bytes) return bad("bytes is NULL");
    *bytes = product_work(o, nullptr).bytes;
    return FT_OK;
  });
}

int ft_moe_int_matmul(const ft_moe_int_product* desc, const int8_t* x, const float* x_scale, const int8_t* w,
                      const float* w_scale, void* y, void* work, int64_t work_bytes, void* hip_stream) {
  return guarded([&]() -> int {
    ft_moe_int_product d;
    if (const int rc = check_product(desc, d)) return rc;
    if (d.tokens == 0) return FT_OK;
    const ProductWork k = product_work(d, work, x, w);
    const int64_t need = k.bytes;
    if (const int rc = check_work(work, work_bytes, need)) return rc;
    if (same(y, {x, x_scale, w, w_scale, work}) || (need && same(work, {x, x_scale, w, w_scale})))
      return bad("an output is also another argument");
    const hipStream_t s = static_cast<hipStream_t>(hip_stream);
    const int64_t es = size_of(d.out_dtype);
    DeviceGuard g;
    if (const int rc = g.enter(s, {{x, 1, "x"}, {x_scale, 4, "x_scale"}, {w, 1, "w"}, {w_scale, 4, "w_scale"}, {y, es, "y"},
                                   {need ? work : y, need ? 16 : es, "work"}}))
      return rc;
    FT_HIP_CHECK(launch_dense_pack(k.packs, s));
    DenseProblem p = product(k.x, k.ld_x, k.w, k.ld_w, d.tokens, d.out, d.in, y, d.ld_y, 1);
    p.a_whole = k.whole_x;
    p.b_whole = k.whole_w;
    p.xs = x_scale;
    p.ws[0] = p.ws[1] = w_scale;
    return run(kDenseInt, d.out_dtype, {p}, k.part, s);
  });
}

int ft_moe_int_gated_ffn_work(const ft_moe_gated_ffn* d, int64_t* bytes) {
  return guarded([&]() -> int {
    ft_moe_gated_ffn o;
    if (const int rc = check_int_ffn(d, o)) return rc;
    if (!bytes) return bad("bytes is NULL");
    *bytes = int_work(o, nullptr).bytes;
    return FT_OK;
  });
}

int ft_moe_int_gated_ffn(const ft_moe_gated_ffn* desc, const void* x, const int8_t* w_gate, const float* gate_scale,
                         const int8_t* w_up, const float* up_scale, const int8_t* w_down, const float* down_scale,
                         void* y, void* work, int64_t work_bytes, void* hip_stream) {
  return guarded([&]() -> int {
    ft_moe_gated_ffn d;
    if (const int rc = check_int_ffn(desc, d)) return rc;
    if (d.tokens == 0) return FT_OK;
    const IntWork w = int_work(d, work, w_gate, w_up, w_down);
    if (const int rc = check_work(work, work_bytes, w.bytes)) return rc;
    if (same(y, {x, w_gate, gate_scale, w_up, up_scale, w_down, down_scale, work}) ||
        same(work, {x, w_gate, gate_scale, w_up, up_scale, w_down, down_scale}))
      return bad("an output is also another argument");
    const hipStream_t s = static_cast<hipStream_t>(hip_stream);
    DeviceGuard g;
    if (const int rc = g.enter(s, {{x, 2, "x"}, {w_gate, 1, "w_gate"}, {gate_scale, 4, "gate_scale"}, {w_up, 1, "w_up"},
                                   {up_scale, 4, "up_scale"}, {w_down, 1, "w_down"}, {down_scale, 4, "down_scale"},
                                   {y, 2, "y"}, {work, 16, "work"}}))
      return rc;
    const int T = d.tokens, H = d.hidden, I = d.inter;
    FT_HIP_CHECK(launch_dense_pack(w.packs, s));
    DenseProblem p = product(w.xq, w.ldx, w.wg, w.ld_in, T, I, H, w.h, w.ldf, 1);
    p.b[1] = u8(w.wu);
    p.a_whole = w.whole_x;
    p.b_whole = w.whole_in;
    p.xs = w.xs;
    p.ws[0] = gate_scale;
    p.ws[1] = up_scale;
    if (const int rc = run_quantized(kDenseIntGated, FT_DT_F32, p, d.dtype, x, d.ld_x, w.part, s)) return rc;
    p = product(w.hq, w.ldh, w.wd, w.ld_out, T, H, I, y, d.ld_y, 1);
    p.a_whole = w.whole_h;
    p.b_whole = w.whole_out;
    p.xs = w.hs;
    p.ws[0] = p.ws[1] = down_scale;
    return run_quantized(kDenseInt, d.dtype, p, FT_DT_F32, w.h, w.ldf, w.part, s);
  });
}

}  // extern "C"
