// The dense products on large tiles: device code, instantiated by the
// dense_tile_*.hip units.
//
// A workgroup owns TM x TN results (TN counts the columns of both matrices in
// a gated form) and walks K in steps of 128 bytes.  Each operand's tile is two
// halves ("units"), lo and hi, and so is each wave's part of the tile: it owns
// the four quadrants lo/hi x lo/hi of its rows and columns in accumulators.
//
// Schedule.  A step is four products, lo x lo, lo x hi, hi x hi, hi x lo (A x
// B), chosen so that each unit is read from LDS once, one product ahead of its
// use, into registers.  Its LDS slot is free from then on, and the load of the
// same unit two steps later starts at once: with two slots per unit (128 KB for
// 256 x 256) three halves of a step are always in flight, 1.5 steps ahead of
// their use.  One barrier per half step makes a half's loads visible (vmcnt of
// everything older than the two latest halves) and frees the slots read in
// the half before.  Reads and loads are spread between the matrix
// instructions.  With the reads of a step in K order, whose slots are free only
// at its end, 8192^3 ran at 1.09 to 1.14 PFLOP/s, so at 1.24 (32x32 instructions).
//
// Loads.  buffer_load ... lds moves 16 bytes per lane straight into LDS, lane
// i at + 16 i of a uniform address: 1 KB per instruction.  An operand along K
// is staged as rows of 128 bytes (8 rows per instruction), one across K as its
// 64 rows of k, a unit's elements wide.  Lanes outside the matrix (rows past
// the end, K past the end) are given an offset beyond the buffer's range, for
// which the load writes zeros, so any size runs without an edge case in the loop.
//
// Bank conflicts.  Units cannot be padded (the loads write contiguously), so
// the 16-byte pieces of a row are permuted instead, on the side of the source
// addresses: row r holds piece c at place c ^ key(r), key(r) distinct for the
// rows that one LDS cycle reads.  SQ_LDS_BANK_CONFLICT counts none for operands
// along K; across K the reads of B meet each bank twice (8192 tokens, H 7168, I
// 2048: 7.4 M cycles of all CUs in dh, 36.8 M in dx and the weight gradients).
//
// Operands.  Lane l of a 16x16 matrix instruction needs row l % 16, K bytes
// 16 (l / 16) .. + 15 of a 64-byte step.  Along K that is one 16-byte LDS
// read.  Across K two ds_read_b64_tr_b16 turn 4 (k) x 16 (row) blocks while
// they are read: lane i of each group of 16 gives the address of four rows'
// elements at k = i / 4 and receives row i's four k.  The weights (n) are the
// first operand, so a lane ends with runs of n of one row m.
//
// Bound by the matrix cores at the card's power limit: at 8192^3 the clock
// drops to 1.9 GHz with them busy 75% of the cycles.  The 16x16 instructions
// ran 6% faster than the 32x32 ones (which draw more: 1.65 GHz), eight waves
// 36% faster than four of 128 x 128.  8192^3, sustained: bf16 1.32 PFLOP/s,
// 8 bit 2.16; K across both operands 1.23.  8192 tokens, H 7168, I 2048: forward
// with g and u kept 532 us (1.36 PFLOP/s), backward 1087 us (1.33).  The 256 x 256
// kernels take all 256 registers of a lane and spill some: 20 to 22 in dh, 10 in
// dx with the weight gradients, 1 to 9 in the others; the 128 x 128 ones none.
#pragma once
#include <algorithm>
#include <type_traits>

#include "dense.h"

namespace ftmoe {

#define FT_L3 __attribute__((address_space(3)))

typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr uint32_t kOutside = 0x80000000u;  // an offset beyond every buffer's range
constexpr int kTileKB = 128;                // bytes of K per step

// 16 bytes per lane from buffer r at off to LDS offset lds + 16 * lane
// (lds uniform); lanes outside the buffer's range write zeros.  Written in
// assembly because the compiler, unable to tell which LDS bytes such a load
// writes, waits for all of them before every transposing read.  It has no
// result register; who reads the LDS bytes waits for vmcnt first.
typedef uint32_t tile_rsrc __attribute__((ext_vector_type(4)));
__device__ __attribute__((always_inline)) inline tile_rsrc tile_buffer(const uint8_t* p, uint32_t bytes) {
  const uint64_t a = uint64_t(uintptr_t(p));
  return tile_rsrc{uint32_t(a), uint32_t(a >> 32) & 0xFFFFu, bytes, 0x00020000u};
}
__device__ __attribute__((always_inline)) inline void tile_load16(tile_rsrc r, uint32_t lds, uint32_t off) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds"
               :
               : "s"(lds), "v"(off), "s"(r)
               : "m0");
}

// LDS keys: the 16-byte pieces of a staged row are permuted, see above.  An
// operand along K has 128-byte rows, two of them side by side over the 256
// bytes of the banks; one LDS cycle of a fragment read takes the 16 rows of 16
// lanes.  B rows are handed out to lanes as n = 8 (r / 4) + 4 t + r % 4 (lane
// row r, fragment t of a pair), so a lane's sums of a pair are 8 neighbours.
__device__ __attribute__((always_inline)) inline int tile_key_a(int r) { return (r >> 1) & 7; }
__device__ __attribute__((always_inline)) inline int tile_key_b(int n) { return ((n >> 1) & 1) | ((n >> 3) & 3) << 1; }
// An operand across K: rows of R elements of one k; one LDS cycle of a
// transposing read takes 32 bytes of the rows k = 0..3 and 8..11 (+ 4, + 16).
template <int R>
__device__ __attribute__((always_inline)) inline int tile_key_cols(int k) {
  return R >= 128 ? ((k & 3) | ((k >> 3) & 1) << 2) << 1 : (((k >> 1) & 1) | ((k >> 3) & 1) << 1) << 1;
}

// One operand: halves (units) of R rows, loaded by NW waves.
template <bool ROWS, bool IS_B, int R, int NW, int ES>
struct TileOperand {
  static constexpr int kUnit = R * kTileKB;        // bytes of a staged unit
  static constexpr int kPer = kUnit / 1024 / NW;   // load instructions per wave and unit
  static constexpr int KE = kTileKB / ES;
  static constexpr int kPieces = R / 8;            // !ROWS: 16-byte pieces of a k row
  static_assert(kPer * NW * 1024 == kUnit, "whole instructions per wave");
  uint32_t row;         // this lane's staged row (ROWS: of the unit, else k) in load 0
  uint32_t edge[kPer];  // ROWS: the piece's byte in the 128 of its row; else in the k row

  __device__ __attribute__((always_inline)) inline void init(int w, int lane) {
    row = ROWS ? uint32_t(w * kPer * 8 + (lane >> 3)) : uint32_t((w * kPer * 64 + lane) / kPieces);
#pragma unroll
    for (int q = 0; q < kPer; ++q) {
      const int r = int(row) + q * (ROWS ? 8 : 64 / kPieces);
      edge[q] = ROWS ? uint32_t((lane & 7) ^ (IS_B ? tile_key_b(r) : tile_key_a(r))) * 16
                     : uint32_t((lane % kPieces) ^ tile_key_cols<R>(r)) * 16;
    }
  }
  // load instruction q of a unit whose first row (column) lies at p and has
  // `rows` rows (columns) from there on; `elems` elements of K from p on
  __device__ __attribute__((always_inline)) inline void load(const uint8_t* p, int64_t ld, int rows, int elems, uint32_t dst,
                                                             int w, int q) const {
    dst += uint32_t(w * kPer + q) * 1024;
    const uint32_t r = row + uint32_t(q * (ROWS ? 8 : 64 / kPieces));
    const uint32_t off = r * uint32_t(ld) + edge[q];
    if constexpr (ROWS) {
      const int64_t bytes = int64_t(max(rows, 0)) * ld;
      const auto buf = tile_buffer(p, uint32_t(min(bytes, int64_t(0x7FFFFFFF))));
      tile_load16(buf, dst, edge[q] < uint32_t(elems * ES) ? off : kOutside);
    } else {
      const auto buf = tile_buffer(p, uint32_t(elems) * uint32_t(ld));
      tile_load16(buf, dst, int(edge[q]) < rows * ES ? off : kOutside);
    }
  }
};

template <typename D, int FORM, typename TO, int TM, int TN, int WM, int WN, bool LO = false>
struct TileKernel {
  typedef typename D::elem E;
  typedef typename D::acc4 Acc;
  static constexpr bool AR = dense_a_rows(FORM), BR = dense_b_rows(FORM), TWO = dense_two_b(FORM);
  static constexpr int NW = WM * WN, ES = int(sizeof(E)), KE = kTileKB / ES;
  static constexpr int HM = TM / 2, HN = TN / 2;             // rows of a unit
  static constexpr int MF = HM / WM / 16, NF = HN / WN / 16; // fragments of a wave per unit
  static constexpr int KS = kTileKB / 64;                    // matrix instructions along K per step
  static constexpr int NOUT = TWO ? HN : TN;                 // output columns of a tile
  // A's second half holds what the rounding of the first half's rows left off: the same
  // lanes end with the sums of both, which are added (64 tokens, H 2048, I 768: backward
  // 30.8 us, as without; as rows of their own, joined in memory, 32.8)
  static constexpr bool kFold = LO && FORM == kDenseCols;
  static constexpr int kRows = kFold ? MF : 2 * MF;          // rows of a lane's results
  typedef TileOperand<AR, false, HM, NW, ES> OA;
  typedef TileOperand<BR, true, HN, NW, ES> OB;
  // LDS: two of each unit: A lo, A hi, B lo, B hi
  static constexpr int kLds = 2 * (2 * OA::kUnit + 2 * OB::kUnit);
  static_assert(NF % 2 == 0, "B rows are handed out to pairs of fragments");
  static_assert(AR == BR || ES == 2, "8-bit operands lie along K");

  static __device__ __attribute__((always_inline)) inline int at_a(int par, int half) { return (par * 2 + half) * OA::kUnit; }
  static __device__ __attribute__((always_inline)) inline int at_b(int par, int half) {
    return (par * 2 + half) * OB::kUnit;  // from the first B unit, 4 A units in
  }

  struct FragA { u32x4 v[MF][KS]; };
  struct FragB { u32x4 v[NF][KS]; };

  // LDS addresses of a lane's fragment reads within a unit, one per value that
  // a constant offset does not reach (the pieces' places are permuted): along
  // K by K step, for B by fragment of a pair too; across K by fragment
  static constexpr int kAddrA = AR ? KS : MF, kAddrB = BR ? KS : NF;
  static __device__ __attribute__((always_inline)) inline uint32_t addr_rows(int row0, int lane, int ks, bool is_b) {
    const int r = lane & 15, row = is_b ? 8 * (r >> 2) + (r & 3) : r;
    return uint32_t((row0 + row) * kTileKB + (((4 * ks + (lane >> 4)) ^ (r >> 1)) * 16));
  }
  // B fragments come in pairs there too: fragment t of a pair takes the columns
  // 8 c + 4 t .. + 3, c = 0..3 (its reads then meet each bank twice)
  template <int R>
  static __device__ __attribute__((always_inline)) inline uint32_t addr_cols(int row0, int lane, bool pairs) {
    const int i = lane & 15, m = row0 + (i & 3) * (pairs ? 8 : 4), k = 8 * (lane >> 4) + (i >> 2);
    return uint32_t(k * (R * 2) + (((m >> 3) ^ tile_key_cols<R>(k)) * 16) + (m & 7) * 2);
  }
  static __device__ __attribute__((always_inline)) inline u32x4 lds_rows(uint32_t at) {
    return *(FT_L3 const u32x4*)at;
  }
  template <int R>
  static __device__ __attribute__((always_inline)) inline u32x4 lds_cols(uint32_t at) {
    const s16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((FT_L3 s16x4*)at);
    const s16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((FT_L3 s16x4*)(at + 4 * R * 2));
    typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
    const u32x2 l = (u32x2)lo, h = (u32x2)hi;
    return u32x4{l[0], l[1], h[0], h[1]};
  }
  // read q of a unit's fragments, K steps outermost; unit: its byte offset
  static __device__ __attribute__((always_inline)) inline void read_a(FragA& f, const uint32_t (&at)[kAddrA], int unit, int q) {
    const int ks = q / MF, i = q % MF;
    if constexpr (AR)
      f.v[i][ks] = lds_rows(at[ks] + unit + i * 16 * kTileKB);
    else
      f.v[i][ks] = lds_cols<HM>(at[i] + unit + ks * 32 * HM * 2);
  }
  static __device__ __attribute__((always_inline)) inline void read_b(FragB& f, const uint32_t (&at)[kAddrB], int unit, int q) {
    const int ks = q / NF, j = q % NF;
    if constexpr (BR)
      f.v[j][ks] = lds_rows(at[ks] + unit + ((j / 2) * 32 + (j % 2) * 4) * kTileKB);
    else
      f.v[j][ks] = lds_cols<HN>(at[j] + unit + ks * 32 * HN * 2);
  }

  // Where one workgroup's piece of work (a tile, and a part of K) lies.
  struct Place {
    const uint8_t *a[2], *b[2];  // by K segment, or by matrix (TWO); at the tile's first row
    int64_t lda, ldb;
    int rows_a, rows_b;          // from the tile's first
    int k, per, segs;            // elements and steps of a segment
    int first, count;            // K steps of this part
    int m0, n0, problem, split;
  };
  static __device__ __attribute__((always_inline)) inline Place place(const DenseLaunch& l, int item) {
    Place o;
    o.split = item / l.tiles;
    item -= o.split * l.tiles;
    int pi = 0, tm = 0, tn = 0;
    for (;; ++pi) {
      tm = (l.p[pi].m + TM - 1) / TM;
      tn = (l.p[pi].n + NOUT - 1) / NOUT;
      if (item < tm * tn || pi == l.count - 1) break;
      item -= tm * tn;
    }
    const DenseProblem& p = l.p[pi];
    // down blocks of kGroup row tiles
    constexpr int kGroup = 8;
    const int grp = item / (kGroup * tn), in = item - grp * kGroup * tn;
    const int gh = min(kGroup, tm - grp * kGroup);
    o.problem = pi;
    o.m0 = (grp * kGroup + in % gh) * TM;
    o.n0 = in / gh * NOUT;
    o.lda = p.lda;
    o.ldb = p.ldb;
    o.rows_a = (kFold ? p.m + HM : p.m) - o.m0;
    o.rows_b = p.n - o.n0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      o.a[i] = p.a[i] + (AR ? int64_t(o.m0) * p.lda : int64_t(o.m0) * ES);
      o.b[i] = p.b[i] + (BR ? int64_t(o.n0) * p.ldb : int64_t(o.n0) * ES);
    }
    o.k = p.k;
    o.per = (p.k + KE - 1) / KE;
    o.segs = p.segs;
    const int all = o.per * p.segs;
    o.first = int(int64_t(all) * o.split / l.splits);
    o.count = int(int64_t(all) * (o.split + 1) / l.splits) - o.first;
    return o;
  }

  // XCD x (workgroups are dealt to the eight in turn by their number) takes
  // the contiguous range x of the items, so the tiles it works on at a time
  // share rows of A and of B in its L2.
  static __device__ __attribute__((always_inline)) inline int range(const DenseLaunch& l, int xcd) {
    return int(int64_t(l.tiles) * l.splits * xcd / 8);
  }

  // Runs items `item`, next(item), ... below `end`; returns the first that is not.
  template <typename NEXT>
  static __device__ __attribute__((always_inline)) inline int run(const DenseLaunch& l, uint8_t* lds, int item, int end,
                                                                  NEXT next) {
    const int lane = threadIdx.x & 63;
    const int w = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
    const int wm = w % WM, wn = w / WM;
    OA oa;
    OB ob;
    oa.init(w, lane);
    ob.init(w, lane);
    const uint32_t lds0 = uint32_t(uintptr_t((FT_L3 uint8_t*)lds));
    // load instruction q of a unit of step `at` of a place; beyond its steps, zeros
    auto load_a = [&](const Place& o, int at, int par, int half, int q) {
      const int s = o.first + at, seg = o.segs > 1 && s >= o.per ? 1 : 0, kb = s - seg * o.per;
      const int elems = at < o.count ? min(o.k - kb * KE, KE) : 0;
      const int64_t step = int64_t(kb) * (AR ? int64_t(kTileKB) : KE * o.lda);
      oa.load(o.a[seg] + step + half * HM * (AR ? o.lda : int64_t(ES)), o.lda, o.rows_a - half * HM, elems,
              lds0 + at_a(par, half), w, q);
    };
    auto load_b = [&](const Place& o, int at, int par, int half, int q) {
      const int s = o.first + at, seg = o.segs > 1 && s >= o.per ? 1 : 0, kb = s - seg * o.per;
      const int elems = at < o.count ? min(o.k - kb * KE, KE) : 0;
      const int64_t step = int64_t(kb) * (BR ? int64_t(kTileKB) : KE * o.ldb);
      const int first = TWO ? 0 : half * HN;
      ob.load(o.b[TWO ? half : seg] + step + first * (BR ? o.ldb : int64_t(ES)), o.ldb, o.rows_b - first, elems,
              lds0 + 4 * OA::kUnit + at_b(par, half), w, q);
    };

    Acc acc[2][2][MF][NF];  // by halves of A and B
    // the products of one pair of units, with more(e) after product e: what is
    // read and loaded meanwhile is spread between them
    constexpr int kMma = MF * NF * KS, kReadA = MF * KS, kReadB = NF * KS;
    auto mma = [&](Acc (&c)[MF][NF], const FragA& a, const FragB& b, auto more) {
#pragma unroll
      for (int e = 0; e < kMma; ++e) {
        const int ks = e / (MF * NF), i = e / NF % MF, j = e % NF;
        c[i][j] = D::mfma16(b.v[j][ks], a.v[i][ks], c[i][j]);
        more(e);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    auto spread = [&](int e, int count, auto what) {
#pragma unroll
      for (int q = e * count / kMma; q < (e + 1) * count / kMma; ++q) what(q);
    };
    // this wave's LDS reads have ended and all but its latest loads landed; then all waves'
    constexpr int kHalf = OA::kPer + OB::kPer;  // loads of half a step
    auto meet = [&]() {
      asm volatile("" ::: "memory");
      __builtin_amdgcn_s_waitcnt((2 * kHalf) & 0xF | (2 * kHalf) >> 4 << 14 | 0x70);  // vmcnt(2 kHalf) lgkmcnt(0)
      __builtin_amdgcn_s_barrier();
      asm volatile("" ::: "memory");
    };

    uint32_t addr_a[kAddrA], addr_b[kAddrB];
#pragma unroll
    for (int i = 0; i < kAddrA; ++i)
      addr_a[i] = lds0 + (AR ? addr_rows(wm * MF * 16, lane, i, false) : addr_cols<HM>(wm * MF * 16 + i * 16, lane, false));
#pragma unroll
    for (int i = 0; i < kAddrB; ++i)
      addr_b[i] = lds0 + 4 * OA::kUnit +
                  (BR ? addr_rows(wn * NF * 16, lane, i, true) : addr_cols<HN>(wn * NF * 16 + (i / 2) * 32 + i % 2 * 4, lane, true));
    FragA al, ah;
    FragB bx, by;

    // one K step: lo x lo, lo x hi, hi x hi, hi x lo; `lo` holds B lo on entry,
    // `hi` takes B hi and then the next step's B lo.  Loads are those of step
    // `at` of `from`, two steps on.
    auto step = [&](auto parity, FragB& lo, FragB& hi, const Place& from, int at) {
      constexpr int P = decltype(parity)::value;
      meet();  // B hi, A hi of this step are there; the slots of A lo, B lo are free
      mma(acc[0][0], al, lo, [&](int e) {
        spread(e, kReadB, [&](int q) { read_b(hi, addr_b, at_b(P, 1), q); });
        spread(e, OA::kPer, [&](int q) { load_a(from, at, P, 0, q); });
      });
      mma(acc[0][1], al, hi, [&](int e) {
        spread(e, kReadA, [&](int q) { read_a(ah, addr_a, at_a(P, 1), q); });
        spread(e, OB::kPer, [&](int q) { load_b(from, at, P, 0, q); });
      });
      meet();  // A lo, B lo of the next step are there; the slots of B hi, A hi are free
      mma(acc[1][1], ah, hi, [&](int e) {
        spread(e, kReadA, [&](int q) { read_a(al, addr_a, at_a(1 - P, 0), q); });
        spread(e, OB::kPer, [&](int q) { load_b(from, at, P, 1, q); });
      });
      mma(acc[1][0], ah, lo, [&](int e) {
        spread(e, kReadB, [&](int q) { read_b(hi, addr_b, at_b(1 - P, 0), q); });
        spread(e, OA::kPer, [&](int q) { load_a(from, at, P, 1, q); });
      });
    };

    // The pipeline is filled once; behind a tile's last steps it loads and
    // reads the first of the workgroup's next tile.  Steps run in pairs (the
    // LDS slots alternate): an odd count is filled up with a step of zeros.
    Place cur = place(l, item);
    auto fill = [&](int at, int half) {
      if (half == 0) {
#pragma unroll
        for (int q = 0; q < OA::kPer; ++q) load_a(cur, at, at, 0, q);
      }
#pragma unroll
      for (int q = 0; q < OB::kPer; ++q) load_b(cur, at, at, half, q);
      if (half == 1) {
#pragma unroll
        for (int q = 0; q < OA::kPer; ++q) load_a(cur, at, at, 1, q);
      }
    };
    fill(0, 0);
    fill(0, 1);
    fill(1, 0);
    meet();
#pragma unroll
    for (int q = 0; q < kReadA; ++q) read_a(al, addr_a, at_a(0, 0), q);
#pragma unroll
    for (int q = 0; q < kReadB; ++q) read_b(bx, addr_b, at_b(0, 0), q);
    fill(1, 1);

    for (;;) {
      item = next(item);
      const bool last = item >= end;
      Place nxt = last ? cur : place(l, item);
      if (last) nxt.count = 0;
#pragma unroll
      for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int i = 0; i < MF * NF; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[x >> 1][x & 1][i / NF][i % NF][e] = 0;
      int kb = 0;
      for (; kb + 2 < cur.count; kb += 2) {
        step(std::integral_constant<int, 0>(), bx, by, cur, kb + 2);
        step(std::integral_constant<int, 1>(), by, bx, cur, kb + 3);
      }
      step(std::integral_constant<int, 0>(), bx, by, nxt, 0);
      step(std::integral_constant<int, 1>(), by, bx, nxt, 1);
      if constexpr (kFold) {
#pragma unroll
        for (int y = 0; y < 2; ++y)
#pragma unroll
          for (int i = 0; i < MF * NF; ++i) acc[0][y][i / NF][i % NF] += acc[1][y][i / NF][i % NF];
      }
      finish(l, cur, acc, wm, wn, lane);
      if (last) break;
      cur = nxt;
    }
    __builtin_amdgcn_s_waitcnt(0x0070);  // the loads past the end
    return item;
  }

  static __device__ __attribute__((always_inline)) inline void finish(const DenseLaunch& l, const Place& o,
                                                                      const Acc (&acc)[2][2][MF][NF], int wm, int wn,
                                                                      int lane) {
    const DenseProblem& p = l.p[o.problem];
    const int m0 = o.m0, n0 = o.n0, split = o.split;
    // results: lane l has row m = l % 16 of each A fragment and eight columns of each pair of B fragments
    constexpr int YS = TWO ? 1 : 2;
    auto column = [&](int y, int j) { return n0 + (TWO ? 0 : y * HN) + wn * NF * 16 + j * 32 + 8 * (lane >> 4); };
    auto row = [&](int xi) { return int64_t(m0) + (xi / MF) * HM + wm * MF * 16 + xi % MF * 16 + (lane & 15); };
    if (p.part) {
      // the sums of a part of K: whole groups of four (columns past the end hold zeros)
      typedef typename D::sum Sum;
      const int64_t ldp = (p.n + 3) / 4 * 4, mat = int64_t(p.m) * ldp;
      Sum* const s = reinterpret_cast<Sum*>(p.part) + split * (TWO ? 2 : 1) * mat;
#pragma unroll
      for (int xi = 0; xi < kRows; ++xi)
#pragma unroll
        for (int y = 0; y < YS; ++y)
#pragma unroll
          for (int j = 0; j < NF; ++j) {
            const int64_t m = row(xi);
            const int n = column(y, j / 2) + j % 2 * 4;
            if (m >= p.m || n >= p.n) continue;
            gstore<Acc>(s + m * ldp + n, acc[xi / MF][y][xi % MF][j]);
            if constexpr (TWO) gstore<Acc>(s + mat + m * ldp + n, acc[xi / MF][1][xi % MF][j]);
          }
      return;
    }
    // rows of a multiple of eight: whole groups, without a branch around a load
    if (p.n % 8 == 0)
      emit<true>(p, acc, row, column);
    else
      emit<false>(p, acc, row, column);
  }

  // What the sums are combined with is read ahead of the stores: the scales at
  // once, gu some rows ahead (what the registers hold).  WHOLE: columns come in
  // whole groups of eight; reads outside the matrix are moved to its last row
  // and group.
  template <bool WHOLE, typename ROW, typename COLUMN>
  static __device__ __attribute__((always_inline)) inline void emit(const DenseProblem& p, const Acc (&acc)[2][2][MF][NF],
                                                                    ROW row, COLUMN column) {
    constexpr int YS = TWO ? 1 : 2, PF = NF / 2;
    DenseScales<8> ws[YS][PF];
    float xs[kRows];
    constexpr int kAhead = kRows <= 4 ? 3 : 1;
    DenseWith<FORM, E, 8> with[kAhead + 1][YS][PF];
    if constexpr (dense_int(FORM)) {
#pragma unroll
      for (int y = 0; y < YS; ++y)
#pragma unroll
        for (int j = 0; j < PF; ++j) ws[y][j].template fetch<TWO>(p, column(y, j));
#pragma unroll
      for (int xi = 0; xi < kRows; ++xi) xs[xi] = gload<float>(p.xs + min(row(xi), int64_t(p.m) - 1));
    }
    auto fetch = [&](int xi) {
      if constexpr (FORM == kDenseGrad) {
#pragma unroll
        for (int y = 0; y < YS; ++y)
#pragma unroll
          for (int j = 0; j < PF; ++j)
            if constexpr (WHOLE)
              with[xi % (kAhead + 1)][y][j].fetch(p, min(row(xi), int64_t(p.m) - 1), min(column(y, j), p.n - 8));
            else
              with[xi % (kAhead + 1)][y][j].fetch(p, row(xi), column(y, j), row(xi) < p.m ? min(p.n - column(y, j), 8) : 0);
      }
    };
#pragma unroll
    for (int xi = 0; xi < kAhead; ++xi) fetch(xi);
#pragma unroll
    for (int xi = 0; xi < kRows; ++xi) {
      if (xi + kAhead < kRows) fetch(xi + kAhead);
      const int64_t m = row(xi);
#pragma unroll
      for (int y = 0; y < YS; ++y)
#pragma unroll
        for (int j = 0; j < PF; ++j) {
          const int n = column(y, j), cnt = WHOLE ? 8 : min(p.n - n, 8);
          typename D::sum v0[8], v1[8];
#pragma unroll
          for (int q = 0; q < 8; ++q) {
            v0[q] = acc[xi / MF][y][xi % MF][2 * j + q / 4][q % 4];
            v1[q] = acc[xi / MF][1][xi % MF][2 * j + q / 4][q % 4];
          }
          if (m >= p.m || n >= p.n) continue;
          if constexpr (dense_int(FORM))
            dense_emit<FORM, TO, 8>(p, m, n, cnt, v0, v1, xs[xi], ws[y][j]);
          else
            dense_emit<FORM, E, TO, 8, LO>(p, m, n, cnt, v0, v1, with[xi % (kAhead + 1)][y][j]);
        }
    }
  }
};

template <typename D, int FORM, typename TO, int TM, int TN, int WM, int WN, bool LO>
__global__ __launch_bounds__(64 * WM * WN, 2) void k_dense_tile(DenseLaunch l) {
  typedef TileKernel<D, FORM, TO, TM, TN, WM, WN, LO> K;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[K::kLds];
  if (l.clear && blockIdx.x == 0 && threadIdx.x < kDenseQueue) gstore<uint32_t>(l.clear + threadIdx.x, 0u);
  // a workgroup takes every (grid / 8)th item of its XCD's range
  const int xcd = int(blockIdx.x) & 7, stride = int(gridDim.x) >> 3;
  const int item = K::range(l, xcd) + (int(blockIdx.x) >> 3), end = K::range(l, xcd + 1);
  if (item < end) K::run(l, lds, item, end, [&](int at) { return at + stride; });
}

template <typename D, int TM, int TN, int WM, int WN, bool LO>
__global__ __launch_bounds__(64 * WM * WN, 2) void k_dense_pair(DensePair l) {
  typedef typename D::elem E;
  typedef TileKernel<D, kDenseOuter, E, TM, TN, WM, WN> O;
  typedef TileKernel<D, kDenseCols, E, TM, TN, WM, WN, LO> C;
  static_assert(O::kLds == C::kLds, "one LDS layout");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[O::kLds];
  __shared__ int taken;
  // items of this XCD: the weight gradients' tiles, then dx's
  const int xcd = int(blockIdx.x) & 7, o0 = O::range(l.outer, xcd), no = O::range(l.outer, xcd + 1) - o0;
  const int c0 = C::range(l.cols, xcd), nc = C::range(l.cols, xcd + 1) - c0;
  const int first = int(gridDim.x) >> 3;  // the items that workgroups start with
  auto next = [&](int) {
    __syncthreads();  // everyone has read the one before
    if (threadIdx.x == 0) taken = first + int(atomicAdd(l.queue + xcd, 1u));
    __syncthreads();
    return __builtin_amdgcn_readfirstlane(taken);
  };
  int item = int(blockIdx.x) >> 3;
  if (item < no) item = O::run(l.outer, lds, o0 + item, o0 + no, [&](int at) { return o0 + next(at); }) - o0;
  if (item < no + nc) {
    __syncthreads();  // the weight gradients' LDS reads are over
    C::run(l.cols, lds, c0 + item - no, c0 + nc, [&](int at) { return c0 - no + next(at); });
  }
}

template <int FORM, int TM, int TN>
int64_t count_tiles(const DenseLaunch& l) {
  constexpr int NOUT = dense_two_b(FORM) ? TN / 2 : TN;
  int64_t tiles = 0;
  for (int i = 0; i < l.count; ++i) tiles += int64_t((l.p[i].m + TM - 1) / TM) * ((l.p[i].n + NOUT - 1) / NOUT);
  return tiles;
}

template <typename D, int TM, int TN, int WM, int WN, bool LO = false>
hipError_t launch_pair(DensePair l, hipStream_t s) {
  const int64_t to = count_tiles<kDenseOuter, TM, TN>(l.outer), tc = count_tiles<kDenseCols, TM, TN>(l.cols);
  if (to + tc > (1 << 30) || l.outer.splits != 1 || l.cols.splits != 1) return hipErrorInvalidValue;
  l.outer.tiles = int32_t(to);
  l.cols.tiles = int32_t(tc);
  // each XCD's range is rounded, so the most of one is a tile more than its share
  const int64_t most = 256 * (TM + TN > 256 ? 1 : 2);
  const uint32_t grid = uint32_t(std::min(most, ((to + 7) / 8 + (tc + 7) / 8) * 8));
  hipLaunchKernelGGL((k_dense_pair<D, TM, TN, WM, WN, LO>), dim3(grid), dim3(64 * WM * WN), 0, s, l);
  return hipGetLastError();
}

template <typename D>
hipError_t launch_pairs(int tile, const DensePair& l, hipStream_t s) {
  const DenseProblem& dx = l.cols.p[0];
  if (!dx.a_lo) return tile == 256 ? launch_pair<D, 256, 256, 2, 4>(l, s) : launch_pair<D, 128, 128, 2, 2>(l, s);
  if (tile != 128 || dx.m > 64 || dx.a_lo != 64) return hipErrorInvalidValue;
  return launch_pair<D, 128, 128, 2, 2, true>(l, s);
}

template <typename D, int FORM, typename TO, int TM, int TN, int WM, int WN, bool LO = false>
hipError_t launch_tile(DenseLaunch l, hipStream_t s) {
  typedef TileKernel<D, FORM, TO, TM, TN, WM, WN> K;
  const int64_t tiles = count_tiles<FORM, TM, TN>(l);
  if (tiles == 0) return hipSuccess;
  if (tiles * l.splits > (1 << 30)) return hipErrorInvalidValue;
  l.tiles = int32_t(tiles);
  // as many workgroups as run at a time: one per CU, or two of the small ones
  const int64_t most = 256 * (K::kLds <= 65536 ? 2 : 1);
  const uint32_t grid = uint32_t(std::min(most, (tiles * l.splits + 7) / 8 * 8));
  hipLaunchKernelGGL((k_dense_tile<D, FORM, TO, TM, TN, WM, WN, LO>), dim3(grid), dim3(64 * WM * WN), 0, s, l);
  return hipGetLastError();
}

// The parts' sums added in order, then what the form makes of them.  Bound by
// the reads of the parts.
template <typename D, int FORM, typename TO>
__global__ __launch_bounds__(256) void k_dense_join(DenseLaunch l) {
  typedef typename D::acc4 Acc;
  constexpr bool TWO = dense_two_b(FORM);
  const DenseProblem& p = l.p[blockIdx.y];
  const int64_t ldp = (p.n + 3) / 4 * 4, mat = int64_t(p.m) * ldp;
  const int64_t at = (int64_t(blockIdx.x) * 256 + threadIdx.x) * 4;
  if (at >= mat) return;
  const typename D::sum* s = reinterpret_cast<const typename D::sum*>(p.part) + at;
  // eight parts are read at a time, and added in order
  constexpr int kAhead = 8;
  Acc v0 = {0, 0, 0, 0}, v1 = {0, 0, 0, 0};
  for (int i = 0; i < l.splits; i += kAhead) {
    Acc a[kAhead], b[kAhead];
#pragma unroll
    for (int q = 0; q < kAhead; ++q) {
      a[q] = b[q] = Acc{0, 0, 0, 0};
      if (i + q < l.splits) {
        a[q] = gload<Acc>(s + (i + q) * (TWO ? 2 : 1) * mat);
        if constexpr (TWO) b[q] = gload<Acc>(s + ((i + q) * 2 + 1) * mat);
      }
    }
#pragma unroll
    for (int q = 0; q < kAhead; ++q) v0 += a[q], v1 += b[q];
  }
  const int64_t m = at / ldp;
  const int n = int(at - m * ldp);
  typename D::sum a[4], b[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) a[q] = v0[q], b[q] = v1[q];
  dense_finish<FORM, typename D::elem, TO>(p, m, n, min(p.n - n, 4), a, b);
}

template <typename D, int FORM, typename TO>
hipError_t launch_tiles(int tile, const DenseLaunch& l, hipStream_t s) {
  hipError_t e = hipErrorInvalidValue;
  const DenseProblem& p = l.p[0];
  if (!p.c_lo && !p.a_lo)
    e = tile == 256 ? launch_tile<D, FORM, TO, 256, 256, 2, 4>(l, s) : launch_tile<D, FORM, TO, 128, 128, 2, 2>(l, s);
  else if constexpr (FORM == kDenseGrad || FORM == kDenseCols)  // few tokens: kernels of their own, for the others' registers
    if (tile == 128 && l.count == 1 && p.m <= 64 && p.a_lo == (FORM == kDenseCols ? 64 : 0))
      e = launch_tile<D, FORM, TO, 128, 128, 2, 2, true>(l, s);
  if (e != hipSuccess || l.splits == 1) return e;
  int64_t most = 0;
  for (int i = 0; i < l.count; ++i) most = std::max(most, int64_t(l.p[i].m) * ((l.p[i].n + 3) / 4));
  if (most == 0) return hipSuccess;
  hipLaunchKernelGGL((k_dense_join<D, FORM, TO>), dim3(uint32_t((most + 255) / 256), l.count), dim3(256), 0, s, l);
  return hipGetLastError();
}

}  // namespace ftmoe
