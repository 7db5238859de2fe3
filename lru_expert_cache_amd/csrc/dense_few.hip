// Dense products of few tokens (up to 64) with operands along K: decode.
//
// Bound by reading the weights once.  A workgroup owns 16 FT weight rows (in a
// gated form 8 FT of each matrix) and all tokens; its waves cut K between them
// in turns of 128 bytes, so together they read whole runs of each row.  Each
// wave streams its turns through three LDS stages of its own (no barrier in
// the loop): buffer_load ... lds reads 8 rows x 128 bytes per instruction, whole
// lines, with a row's 16-byte pieces permuted so that the fragment reads (lane
// l: row l % 16, bytes 16 (l / 16) .. of a 64-byte step) meet no bank twice.
// Two stages are in flight while one is multiplied.  Lanes outside the
// matrices write zeros, as a wave's turn past the end of K does, so every wave
// counts the same loads.  The waves' sums meet in LDS and are added
// in the order of the waves.  No second launch, no scratch memory.
//
// Loading fragments straight into registers instead touches 16 lines per
// quarter of a wave: 14.0 us against 9.7 for a gated product of 16 tokens, H
// 6144, I 2048 (50 MB: 5.2 TB/s, a large copy moves 4.9).
//
// Up to 16 tokens of the 16-bit block's h keep what their rounding left off
// (a_lo): as many rows again, 8 or 16 behind, whose sums are added before the
// waves' meet.  Both products of a block, 1 token, H 2048, I 768 6.5 us without,
// 6.9 with; 16 tokens, H 6144, I 2048 16.2 and 16.9.
//
// Eight waves up to 16 rows, four above (their LDS stages are larger; eight
// with two stages: 14.3 us against 14.1 at 64 tokens).  FT is 1 while the
// workgroups then fit the CUs in one round, else 2, which reads the tokens
// half as often: N 6144, K 2048, 16 tokens 6.8 us against 10.0; N 2048 (gated),
// K 6144 10.3 against 9.7.
//
// 8-bit forms quantise up to 16 tokens themselves while the codes fit 16 KB:
// every workgroup reads all the tokens and forms the same codes, which saves a
// launch.  The whole 8-bit block, H 2048, I 768, one token: 9.6 us, with launches
// of their own 14.9; H 7168, I 2048, one token 13.9 and 17.2, 8 tokens 17.2 and
// 17.8.  With 32 KB of codes 16 tokens of the latter took 19.3 us against 18.0.
#include "dense_tile.h"
#include "int_quant.h"

namespace ftmoe {

namespace {

// Tokens that the kernel quantises itself (TX: their type): R of them (a power
// of two up to 16), their codes in LDS as R rows of 128 bytes a unit.  A row
// belongs to 512 / R threads, which keep kTokenPieces pieces of it each.
constexpr int kTokenCodes = 16384;  // bytes, see above
template <typename TX>
constexpr int kTokenPieces = kTokenCodes / 512 / RowPiece<TX>::N;

template <typename TX>
struct TokenCodes {
  int shift;  // log2 R
  __device__ __attribute__((always_inline)) inline explicit TokenCodes(int m) : shift(m > 1 ? 32 - __clz(m - 1) : 0) {}
  // the codes of unit u's row r, 16 bytes at piece c of its 128
  __device__ __attribute__((always_inline)) inline uint32_t at(int u, int r, int c) const {
    return uint32_t(((u << shift) + r) * kTileKB + ((c ^ ((r >> 1) & 7)) * 16));
  }
  // meanwhile() runs once the tokens are there
  template <typename F>
  __device__ __attribute__((always_inline)) inline void fill(const DenseProblem& p, uint8_t* codes, uint32_t* top,
                                                             float* scale, F meanwhile) const {
    constexpr int N = RowPiece<TX>::N, G = kTokenPieces<TX>;
    const int tid = threadIdx.x, per = 512 >> shift, r = tid >> (9 - shift), j = tid & (per - 1);
    const int pieces = (p.k + kTileKB - 1) / kTileKB * kTileKB / N;
    RowPiece<TX> v[G], end;
    RowMax<TX> most;
    // rows past the last token stay zeros
    const int cols = r < p.m ? p.k : 0, whole = p.k / N;
    const TX* x = reinterpret_cast<const TX*>(p.a[0] + min(r, p.m - 1) * p.lda);
    const bool last = whole * N < cols && j == 0;  // has the piece that the row ends in
#pragma unroll
    for (int g = 0; g < G; ++g) v[g].load(x, (j + g * per) * N, cols);
    if (last) {
      end.load_last(x, cols);
      most.add(end);
    }
    if (tid < 16) top[tid] = 0;
    __syncthreads();
#pragma unroll
    for (int g = 0; g < G; ++g) most.add(v[g]);
    uint32_t mx = most.bits();
    asm volatile("" : "+v"(mx)::"memory");
    meanwhile();
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) mx = max(mx, uint32_t(__shfl_xor(int(mx), o)));
    if ((tid & 31) == 0) atomicMax(top + r, mx);  // the largest, whatever the order
    __syncthreads();
    const RowScale q(top[r]);
    if (j == 0) scale[r] = q.scale;
    auto put = [&](int c, const RowPiece<TX>& t) {
      const int e = c * N;
      uint32_t b[N / 4];
      q.codes(t, b);
      uint32_t* to = reinterpret_cast<uint32_t*>(codes + at(e / kTileKB, r, e % kTileKB / 16) + e % 16);
#pragma unroll
      for (int i = 0; i < N / 4; ++i) to[i] = b[i];
    };
#pragma unroll
    for (int g = 0; g < G; ++g) {
      const int c = j + g * per;
      if (c < pieces && (c != whole || whole * N == cols)) put(c, v[g]);
    }
    if (last) put(whole, end);
    __syncthreads();
  }
};

// FT: weight fragments of 16 rows (a gated form: both matrices together); XI:
// load instructions of 8 tokens, 0: the tokens have type TX and are quantised here
template <typename D, int FORM, typename TO, int FT, int XI, int kWaves, typename TX = int8_t>
__global__ __launch_bounds__(64 * kWaves) void k_dense_few(DenseLaunch l) {
  typedef typename D::elem E;
  typedef typename D::acc4 Acc;
  typedef typename D::sum Sum;
  constexpr bool TWO = dense_two_b(FORM);
  constexpr int F = FT * (TWO ? 8 : 16);     // output columns
  constexpr bool QUANT = XI == 0;
  static_assert(!QUANT || kWaves == 8, "512 threads share the tokens");
  constexpr int MT = QUANT ? 1 : (XI + 1) / 2;  // token fragments of 16
  constexpr int S = QUANT && FT == 1 ? 6 : 3;   // LDS stages of a wave
  constexpr int kLoads = 2 * FT + XI;        // per stage
  constexpr int kStage = (FT + (QUANT ? 0 : MT)) * 2048;
  constexpr int kLd = FT * 16 + 4;           // sums of a token, padded
  constexpr int kSums = kWaves * MT * 16 * kLd * 4;
  constexpr int kLds = kWaves * S * kStage > kSums ? kWaves * S * kStage : kSums;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kLds];
  __shared__ __attribute__((aligned(1024))) uint8_t codes[QUANT ? kTokenCodes : 16];
  __shared__ uint32_t top[16];
  __shared__ float scale[16];

  const DenseProblem& p = l.p[0];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
  const int n0 = int(blockIdx.x) * F;
  const int kb = p.k * int(sizeof(E)), units = (kb + kTileKB - 1) / kTileKB;
  const int rounds = (units + kWaves - 1) / kWaves;
  const int64_t lda = p.lda, ldb = p.ldb;
  const uint8_t *const a0 = p.a[0], *const b0 = p.b[0] + n0 * ldb, *const b1 = p.b[1] + n0 * ldb;
  const int64_t a_bytes = (p.m + p.a_lo) * lda, b_bytes = int64_t(p.n - n0) * ldb;

  // load instruction q: 8 rows of 128 bytes; the pieces of row r are permuted by r / 2
  const int r8 = lane >> 3;
  const uint32_t base = uint32_t(uintptr_t((FT_L3 uint8_t*)lds)) + uint32_t(w) * (S * kStage);
  auto issue = [&](int round, int stage) {
    const int at = (w + round * kWaves) * kTileKB;
    const int left = kb - at;  // bytes of K from this unit's first
    const uint32_t dst = base + uint32_t(stage) * kStage;
#pragma unroll
    for (int q = 0; q < kLoads; ++q) {
      const bool is_x = q >= 2 * FT;
      const int i = is_x ? q - 2 * FT : q, half = i & 1;
      const int piece = (lane & 7) ^ (half * 4 + (r8 >> 1));
      // a gated form's rows: 8 gate, 8 up (FT 1); 16 gate, 16 up
      const int mat = !TWO || is_x ? 0 : FT == 1 ? half : (i >> 1) & 1;
      const int row0 = is_x || !TWO ? i * 8 : FT == 1 ? 0 : (i >> 2) * 16 + half * 8;
      const int64_t ld = is_x ? lda : ldb;
      const int64_t bytes = (is_x ? a_bytes : b_bytes) - at;
      const uint8_t* src = (is_x ? a0 : mat ? b1 : b0) + at;
      const auto buf = tile_buffer(src, uint32_t(bytes < 0 ? 0 : bytes > 0x7FFFFFFF ? 0x7FFFFFFF : bytes));
      tile_load16(buf, dst + q * 1024, piece * 16 < left ? uint32_t(row0 + r8) * uint32_t(ld) + piece * 16 : kOutside);
    }
  };
  auto wait = [&](int round) {  // this round's loads have landed, the round before has been read
    asm volatile("" ::: "memory");
    constexpr int n = (S - 2) * kLoads;
    if (round + S - 1 <= rounds)
      __builtin_amdgcn_s_waitcnt((n & 0xF) | (n >> 4 << 14) | 0x70);
    else
      __builtin_amdgcn_s_waitcnt(0x0070);
    asm volatile("" ::: "memory");
  };

  Acc acc[FT][MT];
#pragma unroll
  for (int f = 0; f < FT; ++f)
#pragma unroll
    for (int t = 0; t < MT; ++t) acc[f][t] = Acc{0, 0, 0, 0};
  uint32_t at[2];
#pragma unroll
  for (int s = 0; s < 2; ++s) at[s] = base + (lane & 15) * kTileKB + (((4 * s + (lane >> 4)) ^ ((lane >> 1) & 7)) * 16);
  constexpr int kGroups = F / 4;  // of columns; a thread ends with group threadIdx.x % kGroups
  DenseScales<4> ws;
  if constexpr (dense_int(FORM)) ws.template fetch<TWO>(p, n0 + int(threadIdx.x) % kGroups * 4);
#pragma unroll
  for (int s = 0; s < 2; ++s)
    if (s < rounds) issue(s, s);
  const TokenCodes<TX> tokens(p.m);
  if constexpr (QUANT)  // the tokens' loads wait for all before them, so not all weights' are before them
    tokens.fill(p, codes, top, scale, [&]() {
#pragma unroll
      for (int s = 2; s < S - 1; ++s)
        if (s < rounds) issue(s, s);
    });
  const uint32_t codes0 = uint32_t(uintptr_t((FT_L3 uint8_t*)codes));
  int stage = 0, fill = S - 1;
  for (int i = 0; i < rounds; ++i) {
    wait(i);
    if (i + S - 1 < rounds) issue(i + S - 1, fill);
    u32x4 fw[FT][2], fx[MT][2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
      for (int f = 0; f < FT; ++f) fw[f][s] = *(FT_L3 const u32x4*)(at[s] + stage * kStage + f * 2048);
#pragma unroll
      for (int t = 0; t < MT; ++t)
        if constexpr (QUANT)  // past the last unit the weights are zeros
          fx[t][s] = *(FT_L3 const u32x4*)(codes0 + tokens.at(min(w + i * kWaves, units - 1),
                                                              (lane & 15) & ((1 << tokens.shift) - 1), 4 * s + (lane >> 4)));
        else
          fx[t][s] = *(FT_L3 const u32x4*)(at[s] + stage * kStage + (FT + t) * 2048);
    }
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int f = 0; f < FT; ++f)
#pragma unroll
        for (int t = 0; t < MT; ++t) acc[f][t] = D::mfma16(fw[f][s], fx[t][s], acc[f][t]);
    stage = stage + 1 == S ? 0 : stage + 1;
    fill = fill + 1 == S ? 0 : fill + 1;
  }
  if constexpr (FORM == kDenseRows && (XI == 2 || XI == 4))
    if (p.a_lo) {  // (uniform) the sums of what A's rounding left off, 8 rows (XI 4: 16) behind
#pragma unroll
      for (int f = 0; f < FT; ++f)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[f][0][i] += XI == 2 ? __shfl_xor(acc[f][0][i], 8) : acc[f][MT - 1][i];
    }
  __syncthreads();
  Sum* const part = reinterpret_cast<Sum*>(lds);  // [wave][token][kLd]
#pragma unroll
  for (int f = 0; f < FT; ++f)
#pragma unroll
    for (int t = 0; t < MT; ++t)
      *reinterpret_cast<Acc*>(part + ((w * MT + t) * 16 + (lane & 15)) * kLd + f * 16 + (lane >> 4) * 4) = acc[f][t];
  __syncthreads();

  // a thread per token and four columns
  for (int g = threadIdx.x; g < MT * 16 * kGroups; g += 64 * kWaves) {
    const int m = g / kGroups, q = g % kGroups;
    if (m >= p.m) continue;
    const int c0 = !TWO || FT == 1 ? q * 4 : (q >> 2) * 32 + (q & 3) * 4, c1 = FT == 1 ? 8 + q * 4 : c0 + 16;
    const Sum* s = part + m * kLd;
    Acc v0 = *reinterpret_cast<const Acc*>(s + c0), v1 = v0;
    if constexpr (TWO) v1 = *reinterpret_cast<const Acc*>(s + c1);
#pragma unroll
    for (int i = 1; i < kWaves; ++i) {
      s += MT * 16 * kLd;
      v0 += *reinterpret_cast<const Acc*>(s + c0);
      if constexpr (TWO) v1 += *reinterpret_cast<const Acc*>(s + c1);
    }
    const int n = n0 + q * 4, cnt = min(p.n - n, 4);
    Sum s0[4], s1[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) s0[i] = v0[i], s1[i] = v1[i];
    if (cnt <= 0) continue;
    if constexpr (dense_int(FORM))
      dense_emit<FORM, TO, 4>(p, m, n, cnt, s0, s1, QUANT ? scale[m] : gload<float>(p.xs + m), ws);
    else
      dense_finish<FORM, E, TO>(p, m, n, cnt, s0, s1);
  }
}

template <typename D, int FORM, typename TO, int XI, typename TX = int8_t>
hipError_t launch_xi(const DenseLaunch& l, hipStream_t s) {
  constexpr int kWaves = XI <= 2 ? 8 : 4, F = dense_two_b(FORM) ? 8 : 16, kCus = 256;
  const int wgs = (l.p[0].n + F - 1) / F;
  if (wgs <= kCus)
    hipLaunchKernelGGL((k_dense_few<D, FORM, TO, 1, XI, kWaves, TX>), dim3(wgs), dim3(64 * kWaves), 0, s, l);
  else
    hipLaunchKernelGGL((k_dense_few<D, FORM, TO, 2, XI, kWaves, TX>), dim3((wgs + 1) / 2), dim3(64 * kWaves), 0, s, l);
  return hipGetLastError();
}

template <typename D, int FORM, typename TO>
hipError_t launch(const DenseLaunch& l, hipStream_t s) {
  const int tokens = l.p[0].tokens;
  // rows to quantise: x as the caller has it; h in fp32
  if constexpr (FORM == kDenseIntGated) {
    if (tokens == FT_DT_F16) return launch_xi<D, FORM, TO, 0, _Float16>(l, s);
    if (tokens == FT_DT_BF16) return launch_xi<D, FORM, TO, 0, __bf16>(l, s);
  }
  if constexpr (FORM == kDenseInt)
    if (tokens == FT_DT_F32) return launch_xi<D, FORM, TO, 0, float>(l, s);
  if (tokens) return hipErrorInvalidValue;
  const int rows = l.p[0].a_lo ? 2 * l.p[0].a_lo : l.p[0].m;
  if (rows <= 8) return launch_xi<D, FORM, TO, 1>(l, s);
  if (rows <= 16) return launch_xi<D, FORM, TO, 2>(l, s);
  if (rows <= 32) return launch_xi<D, FORM, TO, 4>(l, s);
  return launch_xi<D, FORM, TO, 8>(l, s);
}

}  // namespace

bool dense_few_quantizes(int m, int k) {
  int rows = 1;
  while (rows < m) rows *= 2;
  return m <= 16 && int64_t(rows) * ((k + kTileKB - 1) / kTileKB * kTileKB) <= kTokenCodes;
}

hipError_t launch_dense_few(DenseForm form, int dtype, const DenseLaunch& l, hipStream_t s) {
  if (l.count != 1 || l.p[0].m > kDenseFewRows) return hipErrorInvalidValue;
  if (l.p[0].a_lo && (form != kDenseRows || l.p[0].m > l.p[0].a_lo || (l.p[0].a_lo != 8 && l.p[0].a_lo != 16))) return hipErrorInvalidValue;
  if (l.p[0].tokens && !dense_few_quantizes(l.p[0].m, l.p[0].k)) return hipErrorInvalidValue;
  if (form == kDenseIntGated) return launch<DenseI8, kDenseIntGated, float>(l, s);
  if (form == kDenseInt) {
    if (dtype == FT_DT_F32) return launch<DenseI8, kDenseInt, float>(l, s);
    if (dtype == FT_DT_F16) return launch<DenseI8, kDenseInt, _Float16>(l, s);
    return launch<DenseI8, kDenseInt, __bf16>(l, s);
  }
  const bool f16 = dtype == FT_DT_F16;
  if (form == kDenseGated)
    return f16 ? launch<DenseF16, kDenseGated, _Float16>(l, s) : launch<DenseBf16, kDenseGated, __bf16>(l, s);
  if (form == kDenseRows)
    return f16 ? launch<DenseF16, kDenseRows, _Float16>(l, s) : launch<DenseBf16, kDenseRows, __bf16>(l, s);
  return hipErrorInvalidValue;
}

}  // namespace ftmoe
