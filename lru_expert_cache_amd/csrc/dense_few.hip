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
// matrices write zeros, and turns past the end of K are such loads too, so
// every wave counts the same loads.  The waves' sums meet in LDS and are added
// in the order of the waves.  No second launch, no scratch memory.
//
// Loading fragments straight into registers instead touches 16 lines per
// quarter of a wave: 14.0 us against 9.7 for a gated product of 16 tokens, H
// 6144, I 2048 (50 MB: 5.2 TB/s, a large copy moves 4.9).
//
// Eight waves up to 16 tokens, four above (their LDS stages are larger; eight
// with two stages: 14.3 us against 14.1 at 64 tokens).  FT is 1 while the
// workgroups then fit the CUs in one round, else 2, which reads the tokens
// half as often: N 6144, K 2048, 16 tokens 6.8 us against 10.0; N 2048 (gated),
// K 6144 10.3 against 9.7.
#include "dense_tile.h"

namespace ftmoe {

namespace {

// FT: weight fragments of 16 rows (a gated form: both matrices together); XI:
// load instructions of 8 tokens
template <typename D, int FORM, typename TO, int FT, int XI, int kWaves>
__global__ __launch_bounds__(64 * kWaves) void k_dense_few(DenseLaunch l) {
  typedef typename D::elem E;
  typedef typename D::acc4 Acc;
  typedef typename D::sum Sum;
  constexpr bool TWO = dense_two_b(FORM);
  constexpr int F = FT * (TWO ? 8 : 16);     // output columns
  constexpr int MT = (XI + 1) / 2;           // token fragments of 16
  constexpr int S = 3;                       // LDS stages of a wave
  constexpr int kLoads = 2 * FT + XI;        // per stage
  constexpr int kStage = (FT + MT) * 2048;
  constexpr int kLd = FT * 16 + 4;           // sums of a token, padded
  constexpr int kSums = kWaves * MT * 16 * kLd * 4;
  constexpr int kLds = kWaves * S * kStage > kSums ? kWaves * S * kStage : kSums;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[kLds];

  const DenseProblem& p = l.p[0];
  const int lane = threadIdx.x & 63, w = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
  const int n0 = int(blockIdx.x) * F;
  const int kb = p.k * int(sizeof(E)), units = (kb + kTileKB - 1) / kTileKB;
  const int rounds = (units + kWaves - 1) / kWaves;
  const int64_t lda = p.lda, ldb = p.ldb;
  const uint8_t *const a0 = p.a[0], *const b0 = p.b[0] + n0 * ldb, *const b1 = p.b[1] + n0 * ldb;
  const int64_t a_bytes = p.m * lda, b_bytes = int64_t(p.n - n0) * ldb;

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
  auto wait = [&]() {  // this round's loads have landed, the round before has been read
    asm volatile("" ::: "memory");
    constexpr int n = (S - 2) * kLoads;
    __builtin_amdgcn_s_waitcnt((n & 0xF) | (n >> 4 << 14) | 0x70);
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
#pragma unroll
  for (int s = 0; s < S - 1; ++s) issue(s, s);
  int stage = 0, fill = S - 1;
  for (int i = 0; i < rounds; ++i) {
    wait();
    issue(i + S - 1, fill);
    u32x4 fw[FT][2], fx[MT][2];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
      for (int f = 0; f < FT; ++f) fw[f][s] = *(FT_L3 const u32x4*)(at[s] + stage * kStage + f * 2048);
#pragma unroll
      for (int t = 0; t < MT; ++t) fx[t][s] = *(FT_L3 const u32x4*)(at[s] + stage * kStage + (FT + t) * 2048);
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
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0070);  // the loads past the end
  __syncthreads();
  Sum* const part = reinterpret_cast<Sum*>(lds);  // [wave][token][kLd]
#pragma unroll
  for (int f = 0; f < FT; ++f)
#pragma unroll
    for (int t = 0; t < MT; ++t)
      *reinterpret_cast<Acc*>(part + ((w * MT + t) * 16 + (lane & 15)) * kLd + f * 16 + (lane >> 4) * 4) = acc[f][t];
  __syncthreads();

  // a thread per token and four columns
  constexpr int kGroups = F / 4;
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
    if (cnt > 0) dense_finish<FORM, E, TO>(p, m, n, cnt, s0, s1);
  }
}

template <typename D, int FORM, typename TO, int XI>
hipError_t launch_xi(const DenseLaunch& l, hipStream_t s) {
  constexpr int kWaves = XI <= 2 ? 8 : 4, F = dense_two_b(FORM) ? 8 : 16, kCus = 256;
  const int wgs = (l.p[0].n + F - 1) / F;
  if (wgs <= kCus)
    hipLaunchKernelGGL((k_dense_few<D, FORM, TO, 1, XI, kWaves>), dim3(wgs), dim3(64 * kWaves), 0, s, l);
  else
    hipLaunchKernelGGL((k_dense_few<D, FORM, TO, 2, XI, kWaves>), dim3((wgs + 1) / 2), dim3(64 * kWaves), 0, s, l);
  return hipGetLastError();
}

template <typename D, int FORM, typename TO>
hipError_t launch(const DenseLaunch& l, hipStream_t s) {
  const int m = l.p[0].m;
  if (m <= 8) return launch_xi<D, FORM, TO, 1>(l, s);
  if (m <= 16) return launch_xi<D, FORM, TO, 2>(l, s);
  if (m <= 32) return launch_xi<D, FORM, TO, 4>(l, s);
  return launch_xi<D, FORM, TO, 8>(l, s);
}

}  // namespace

hipError_t launch_dense_few(DenseForm form, int dtype, const DenseLaunch& l, hipStream_t s) {
  if (l.count != 1 || l.p[0].m > kDenseFewRows) return hipErrorInvalidValue;
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
