// Products of MXFP4 operands: d = a b^T, a [m][k], b [n][k],
//
//   d[i][j] = sum over blocks B of 32 along k of
//             2^(sa[i][B] - 127) 2^(sb[j][B] - 127) sum_{k in B} a[i][k] b[j][k]
//
// dense, by groups of rows (each group of a's rows has a b of its own) and by
// groups along k (each group of columns gives a d of its own).
//
// v_mfma_scale_f32_32x32x64_f8f6f4 takes the codes as they are in memory and a
// scale byte of each operand for each 32 values. Measured here with FP4
// operands it sums to binary32: sums of 64 products are exact while the blocks'
// scales lie within 2^6 of each other (products of two codes are multiples of
// 1/4 up to 36), and 3e-8 off in the 2-norm with scales over 2^20, whatever the
// sum that they enter. A zero code counts as 0 under any scale, subnormal results
// are kept, and scale 255 gives NaN. A sum that leaves binary32's range on the way
// is an infinity. So the accumulators are the instruction's own, and d is rounded
// once at the end.
#include "codec.h"
#include "launch.h"
#include "matmul.h"

namespace nvfp4 {
namespace {

constexpr uint32_t kBlock = kFp8Block;     // values of a row in one block of scales (a word of four)
constexpr uint32_t kBytes = kBlock / 2;    // bytes of a row in one block
constexpr uint32_t kStepBytes = 128;       // bytes of a row in one step along k: two blocks, a cache line

typedef uint32_t u32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

struct Args {
  const uint8_t *a, *b;
  const uint32_t *sa, *sb;  // [kblocks][rows] words
  void *d;
  uint32_t m, n, kblocks;
  uint32_t mode;
  const int32_t *offsets;
  uint32_t groups;
  uint32_t tiles_m, tiles_n;  // of the grid (by groups along k: of one group)
};

// c + the products of 32x32 rows of 64 values; scales in byte SEL of each word.
template <int SEL>
__device__ __forceinline__ f32x16 product32(u32x4 b, u32x4 a, f32x16 c, uint32_t sb, uint32_t sa) {
  typedef int i32x8 __attribute__((ext_vector_type(8)));
  const i32x8 x = __builtin_bit_cast(i32x8, __builtin_shufflevector(b, b, 0, 1, 2, 3, -1, -1, -1, -1));
  const i32x8 y = __builtin_bit_cast(i32x8, __builtin_shufflevector(a, a, 0, 1, 2, 3, -1, -1, -1, -1));
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, y, c, 4, 4, SEL, sb, SEL, sa);
}
// The same of 16x16 rows of 128 values, scales in the lowest byte.
__device__ __forceinline__ f32x4 product16(u32x4 b, u32x4 a, f32x4 c, uint32_t sb, uint32_t sa) {
  typedef int i32x8 __attribute__((ext_vector_type(8)));
  const i32x8 x = __builtin_bit_cast(i32x8, __builtin_shufflevector(b, b, 0, 1, 2, 3, -1, -1, -1, -1));
  const i32x8 y = __builtin_bit_cast(i32x8, __builtin_shufflevector(a, a, 0, 1, 2, 3, -1, -1, -1, -1));
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, 4, 4, 0, sb, 0, sa);
}

// ---------------------------------------------------------------------------
// Tiles of BM x BN, WM x WN waves, each wave (BM / WM) x (BN / WN) in 32x32
// products. A step along k is two blocks, 128 bytes of every row; two stages
// in LDS, filled by loads straight to LDS. KS times as many waves may share a
// tile, each share with every KS-th step, stages and accumulators of its own,
// which are added up at the end.
//
// LDS layout: rows of 128 bytes, eight 16-byte chunks, chunk g of row r at
// place g ^ f(r), so that lanes that read one chunk of neighbouring rows meet
// different banks; the loads to LDS write in lane order, so the permutation
// is in the addresses that they read from. A lane's fragment of a row is one
// chunk: 32 values, one scale.
// The first operand is b, the second a: lane l then holds, for row l % 32 of
// a, rows 8 g + 4 (l / 32) .. + 3, g = 0 .. 3, of the 32x32 tile's b. Which rows
// of b those are is free: tile row 8 g + 4 h + e is row 16 h + 4 g + e, so that a
// lane ends with 16 consecutive columns of d.
// ---------------------------------------------------------------------------
// f(r) of b: with that order of its rows, eight lanes that follow each other get eight values
__device__ __forceinline__ uint32_t swizzle_b(uint32_t r) { return (r & 3) | (r / 16 & 1) << 2; }

template <uint32_t BM, uint32_t BN, uint32_t WM, uint32_t WN, uint32_t KS, bool OUT32>
__global__ __launch_bounds__(WM *WN *KS *kWave) void k_mxfp4_tile(Args p) {
  constexpr uint32_t kWaves = WM * WN;
  constexpr uint32_t TM = BM / WM, TN = BN / WN, MI = TM / 32, NI = TN / 32;
  constexpr uint32_t kLoadA = BM / 8 / kWaves, kLoadB = BN / 8 / kWaves;  // loads of 8 rows that a wave makes
  constexpr uint32_t kGroups = (BM + BN) / 64 * 2, kLoadS = (kGroups + kWaves - 1) / kWaves;  // loads of 64 scale words
  static_assert(TM % 32 == 0 && TN % 32 == 0 && BM % (8 * kWaves) == 0 && BN % (8 * kWaves) == 0 && BM % 64 == 0 && BN % 64 == 0, "tile shape");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[KS][2][(BM + BN) * kStepBytes];
  __shared__ __attribute__((aligned(16))) uint32_t scales[KS][2][2][BM + BN];

  const uint32_t lane = threadIdx.x % kWave, any_wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const uint32_t wave = any_wave % kWaves, share = any_wave / kWaves;  // of the waves that share a tile's steps
  uint32_t tm, tn;
  tile_of(blockIdx.x, p.tiles_n, tm, tn);
  Part part{tm * BM, p.m, 0, p.kblocks, 0, false};
  uint64_t d_base = 0;
  if (p.mode == kGroupedRows) {
    part = find_rows<BM>(p.offsets, p.groups, p.m, p.kblocks, tm);
    if (part.m0 >= part.m_end) return;
  } else if (p.mode == kGroupedK) {
    part.group = tm / p.tiles_m;
    part.m0 = (tm % p.tiles_m) * BM;
    const uint32_t most = p.kblocks * kBlock;
    part.kb0 = clamped(p.offsets[part.group], most) / kBlock;
    part.kb_end = (clamped(p.offsets[part.group + 1], most) + kBlock - 1) / kBlock;
    d_base = static_cast<uint64_t>(part.group) * p.m * p.n;
  }
  const uint32_t m0 = part.m0, n0 = tn * BN;
  const uint64_t pitch = static_cast<uint64_t>(p.kblocks) * kBytes;
  const uint8_t *a = p.a + m0 * pitch, *b = p.b + n0 * pitch;
  const uint32_t *sa = p.sa + m0, *sb = p.sb + n0;
  if (p.mode == kGroupedRows) {
    b += static_cast<uint64_t>(part.group) * p.n * pitch;
    sb += static_cast<uint64_t>(part.group) * p.n * p.kblocks;
  }

  // where this lane's share of each load comes from: rows past the end repeat the last one
  uint32_t from_a[kLoadA], from_b[kLoadB];
#pragma unroll
  for (uint32_t i = 0; i < kLoadA; ++i) {
    const uint32_t r = (wave * kLoadA + i) * 8 + lane / 8;
    from_a[i] = min(r, part.m_end - 1 - m0) * static_cast<uint32_t>(pitch) + ((lane % 8 ^ (r & 7)) << 4);
  }
#pragma unroll
  for (uint32_t i = 0; i < kLoadB; ++i) {
    const uint32_t r = (wave * kLoadB + i) * 8 + lane / 8;
    from_b[i] = min(r, p.n - 1 - n0) * static_cast<uint32_t>(pitch) + ((lane % 8 ^ swizzle_b(r)) << 4);
  }
  const uint32_t last = part.kb_end - 1;
  const uint32_t lds_data = lds_address(&lds[share][0][0]), lds_scales = lds_address(&scales[share][0][0][0]);
  auto load = [&](uint32_t kb, uint32_t stage) {
    const uint8_t *ka = a + static_cast<uint64_t>(kb) * kBytes, *kbp = b + static_cast<uint64_t>(kb) * kBytes;
    const uint32_t to = lds_data + stage * static_cast<uint32_t>(sizeof lds[0][0]);
    // a row's second block where there is none: the first one again, which is not used
    const uint32_t back = kb < last ? 0 : kBytes;
#pragma unroll
    for (uint32_t i = 0; i < kLoadA; ++i) load16_to_lds(to + (wave * kLoadA + i) * 1024, ka, from_a[i] - ((lane % 8 ^ lane / 8) & 4 ? back : 0));
#pragma unroll
    for (uint32_t i = 0; i < kLoadB; ++i)
      load16_to_lds(to + BM * kStepBytes + (wave * kLoadB + i) * 1024, kbp, from_b[i] - ((lane % 8 ^ swizzle_b((wave * kLoadB + i) * 8)) & 4 ? back : 0));
#pragma unroll
    for (uint32_t i = 0; i < kLoadS; ++i) {
      const uint32_t any = (wave * kLoadS + i) % kGroups, w = any % (kGroups / 2), half = any / (kGroups / 2);
      const uint64_t at = min(kb + half, last);
      const bool of_a = w < BM / 64;
      const uint32_t r = (of_a ? w : w - BM / 64) * 64 + lane;
      load4_to_lds(lds_scales + stage * static_cast<uint32_t>(sizeof scales[0][0]) + any * 256, of_a ? sa + at * p.m : sb + at * p.n,
                   4 * min(r, of_a ? part.m_end - 1 - m0 : p.n - 1 - n0));
    }
  };

  const uint32_t wm = wave % WM, wn = wave / WM;
  const uint32_t i32 = lane % 32, h = lane / 32;
  const uint32_t row_b = 16 * (i32 / 4 % 2) + 4 * (i32 / 8) + i32 % 4;
  f32x16 acc[MI][NI];
#pragma unroll
  for (uint32_t i = 0; i < MI; ++i)
#pragma unroll
    for (uint32_t j = 0; j < NI; ++j)
#pragma unroll
      for (uint32_t e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

  // One block: 64 values, then 64 more; a lane's scales of them are bytes h and h + 2 of its rows' words.
  auto block = [&](uint32_t stage, uint32_t half) {
    const uint8_t *la = &lds[share][stage][wm * TM * kStepBytes], *lb = &lds[share][stage][(BM + wn * TN) * kStepBytes];
    const uint32_t *ls = &scales[share][stage][half][wm * TM], *lsb = &scales[share][stage][half][BM + wn * TN];
    uint32_t fa[MI], fb[NI];
#pragma unroll
    for (uint32_t i = 0; i < MI; ++i) fa[i] = ls[32 * i + i32] >> (8 * h);
#pragma unroll
    for (uint32_t j = 0; j < NI; ++j) fb[j] = lsb[32 * j + row_b] >> (8 * h);
#pragma unroll
    for (uint32_t s = 0; s < 2; ++s) {
      const uint32_t chunk = half * 4 + s * 2 + h;
      u32x4 va[MI], vb[NI];
#pragma unroll
      for (uint32_t i = 0; i < MI; ++i) va[i] = *reinterpret_cast<const u32x4 *>(la + (32 * i + i32) * kStepBytes + ((chunk ^ (i32 & 7)) << 4));
#pragma unroll
      for (uint32_t j = 0; j < NI; ++j) vb[j] = *reinterpret_cast<const u32x4 *>(lb + (32 * j + row_b) * kStepBytes + ((chunk ^ swizzle_b(row_b)) << 4));
#pragma unroll
      for (uint32_t i = 0; i < MI; ++i)
#pragma unroll
        for (uint32_t j = 0; j < NI; ++j) acc[i][j] = s == 0 ? product32<0>(vb[j], va[i], acc[i][j], fb[j], fa[i]) : product32<2>(vb[j], va[i], acc[i][j], fb[j], fa[i]);
    }
  };

  if (!part.zero && part.kb0 < part.kb_end) {
    // (a share without a step in the last round loads the last one and leaves it)
    auto first_block = [&](uint32_t kb) { return min(kb, part.kb0 + (last - part.kb0) / 2 * 2); };
    load(first_block(part.kb0 + 2 * share), 0);
    uint32_t stage = 0;
    for (uint32_t first = part.kb0; first < part.kb_end; first += 2 * KS) {
      wait_loads();   // this step's loads are in,
      lds_barrier();  // everyone's are, and everyone has read the other stage
      if (first + 2 * KS < part.kb_end) load(first_block(first + 2 * KS + 2 * share), stage ^ 1);
      const uint32_t kb = first + 2 * share;
      if (kb < part.kb_end) block(stage, 0);
      if (kb + 1 < part.kb_end) block(stage, 1);
      stage ^= 1;
    }
  }

  if (KS > 1) {  // the shares' sums meet in the first one's registers, in their order
    f32x16(*sums)[MI * NI][kWaves][kWave] = reinterpret_cast<f32x16(*)[MI * NI][kWaves][kWave]>(&lds[0][0][0]);
    static_assert((KS - 1) * sizeof sums[0] <= sizeof lds, "the sums fit the stages");
    lds_barrier();
    if (share > 0) {
#pragma unroll
      for (uint32_t i = 0; i < MI; ++i)
#pragma unroll
        for (uint32_t j = 0; j < NI; ++j) sums[share - 1][i * NI + j][wave][lane] = acc[i][j];
    }
    lds_barrier();
    if (share > 0) return;
#pragma unroll
    for (uint32_t k = 0; k + 1 < KS; ++k)
#pragma unroll
      for (uint32_t i = 0; i < MI; ++i)
#pragma unroll
        for (uint32_t j = 0; j < NI; ++j) acc[i][j] += sums[k][i * NI + j][wave][lane];
  }

#pragma unroll
  for (uint32_t i = 0; i < MI; ++i) {
    const uint32_t m = m0 + wm * TM + 32 * i + i32;
    if (m >= part.m_end) continue;
    const uint64_t row = d_base + static_cast<uint64_t>(m) * p.n;
#pragma unroll
    for (uint32_t j = 0; j < NI; ++j) {
      float v[16];
#pragma unroll
      for (uint32_t e = 0; e < 16; ++e) v[e] = acc[i][j][e];
      store<OUT32, 16>(p.d, row, n0 + wn * TN + 32 * j + 16 * h, p.n, v);
    }
  }
}

// ---------------------------------------------------------------------------
// Few rows: tiles of up to kRowsM rows and kRowsN columns, the pairs of blocks
// along k dealt out to the KS waves of a workgroup, each with accumulators of its
// own, which meet in LDS at the end, in the order of the waves. Operands go
// from memory to registers, U pairs of them asked for before the first is used:
// each row of b is read once and by one wave, so LDS would only add a step.
// Lane l's 16 bytes of a block are block l / 16 of four of row l % 16.
// ---------------------------------------------------------------------------
constexpr uint32_t kRowsM = 64, kRowsN = 32;

template <uint32_t KS, uint32_t MT, uint32_t U, bool OUT32>
__device__ __forceinline__ void rows_tile(const Args &p, const Part &part, const uint8_t *a, const uint8_t *b, const uint32_t *sa,
                                          const uint32_t *sb, uint32_t n0, f32x4 (*red)[kRowsM / 16 * 2][kWave]) {
  const uint32_t lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const uint32_t i16 = lane % 16, q = lane / 16;
  const uint32_t pitch = p.kblocks * kBytes;
  // tile t of b takes rows 8 (i / 4) + 4 t + i % 4, so that a lane ends with 8 consecutive columns of d
  uint32_t row_a[MT], row_b[2];
#pragma unroll
  for (uint32_t i = 0; i < MT; ++i) row_a[i] = min(16 * i + i16, part.m_end - 1 - part.m0);
#pragma unroll
  for (uint32_t t = 0; t < 2; ++t) row_b[t] = min(8 * (i16 / 4) + 4 * t + i16 % 4, p.n - 1 - n0);

  f32x4 acc[MT][2];
#pragma unroll
  for (uint32_t i = 0; i < MT; ++i) acc[i][0] = acc[i][1] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  for (uint32_t kb0 = part.kb0 + 2 * wave; kb0 < part.kb_end; kb0 += 2 * U * KS) {
    u32x4 wa[2 * U][MT], wb[2 * U][2];
    uint32_t fa[2 * U][MT], fb[2 * U][2];
#pragma unroll
    for (uint32_t u = 0; u < 2 * U; ++u) {
      const uint32_t kb = min(kb0 + u / 2 * 2 * KS + u % 2, part.kb_end - 1);  // past the end: loaded again, not used
      const uint8_t *ka = a + static_cast<uint64_t>(kb) * kBytes, *kbp = b + static_cast<uint64_t>(kb) * kBytes;
      const uint32_t *ksa = sa + static_cast<uint64_t>(kb) * p.m, *ksb = sb + static_cast<uint64_t>(kb) * p.n;
#pragma unroll
      for (uint32_t t = 0; t < 2; ++t) {
        wb[u][t] = *reinterpret_cast<const u32x4 *>(kbp + row_b[t] * pitch + 16 * q);
        fb[u][t] = ksb[row_b[t]];
      }
#pragma unroll
      for (uint32_t i = 0; i < MT; ++i) {
        wa[u][i] = *reinterpret_cast<const u32x4 *>(ka + row_a[i] * pitch + 16 * q);
        fa[u][i] = ksa[row_a[i]];
      }
    }
#pragma unroll
    for (uint32_t u = 0; u < 2 * U; ++u) {
      if (kb0 + u / 2 * 2 * KS + u % 2 >= part.kb_end) break;
#pragma unroll
      for (uint32_t i = 0; i < MT; ++i)
#pragma unroll
        for (uint32_t t = 0; t < 2; ++t) acc[i][t] = product16(wb[u][t], wa[u][i], acc[i][t], fb[u][t] >> (8 * q), fa[u][i] >> (8 * q));
    }
  }
#pragma unroll
  for (uint32_t i = 0; i < MT; ++i)
#pragma unroll
    for (uint32_t t = 0; t < 2; ++t) red[wave][2 * i + t][lane] = acc[i][t];
  lds_barrier();
  for (uint32_t it = wave; it < 2 * MT; it += KS) {
    f32x4 v = red[0][it][lane];
#pragma unroll
    for (uint32_t w = 1; w < KS; ++w) v += red[w][it][lane];
    const uint32_t m = part.m0 + 16 * (it / 2) + i16;
    if (m < part.m_end) store4<OUT32>(p.d, static_cast<uint64_t>(m) * p.n, n0 + 8 * q + 4 * (it % 2), p.n, v);
  }
}

template <uint32_t KS, bool OUT32>
__global__ __launch_bounds__(KS *kWave) void k_mxfp4_rows(Args p) {
  __shared__ f32x4 red[KS][kRowsM / 16 * 2][kWave];
  const uint32_t tn = blockIdx.x % p.tiles_n, tm = blockIdx.x / p.tiles_n;
  Part part{tm * kRowsM, min(p.m, (tm + 1) * kRowsM), 0, p.kblocks, 0, false};
  if (p.mode == kGroupedRows) {
    part = find_rows<kRowsM>(p.offsets, p.groups, p.m, p.kblocks, tm);
    if (part.m0 >= part.m_end) return;
    part.m_end = min(part.m_end, part.m0 + kRowsM);
    if (part.zero) part.kb_end = 0;
  }
  const uint32_t n0 = tn * kRowsN;
  const uint64_t pitch = static_cast<uint64_t>(p.kblocks) * kBytes;
  const uint8_t *a = p.a + part.m0 * pitch, *b = p.b + n0 * pitch;
  const uint32_t *sa = p.sa + part.m0, *sb = p.sb + n0;
  if (p.mode == kGroupedRows) {
    b += static_cast<uint64_t>(part.group) * p.n * pitch;
    sb += static_cast<uint64_t>(part.group) * p.n * p.kblocks;
  }
  const uint32_t rows = part.m_end - part.m0;
  if (rows <= 16) rows_tile<KS, 1, 4, OUT32>(p, part, a, b, sa, sb, n0, red);
  else if (rows <= 32) rows_tile<KS, 2, 2, OUT32>(p, part, a, b, sa, sb, n0, red);
  else rows_tile<KS, 4, 1, OUT32>(p, part, a, b, sa, sb, n0, red);  // a group's, above the average
}

Args args_of(const Mxfp4Matmul &p, uint32_t bm, uint32_t bn) {
  return Args{p.a, p.b, p.sa, p.sb, p.d, p.m, p.n, p.kblocks, p.mode, p.offsets, p.groups, (p.m + bm - 1) / bm, (p.n + bn - 1) / bn};
}

// The workgroups of tiles of bm rows.
uint64_t tiles_of(const Args &a, uint32_t bm) {
  uint64_t rows = a.tiles_m;
  // every group may end in a partial tile, and so may the rows past the last one
  if (a.mode == kGroupedRows) rows = a.m / bm + a.groups + 1;
  if (a.mode == kGroupedK) rows = static_cast<uint64_t>(a.tiles_m) * a.groups;
  return rows * a.tiles_n;
}

template <uint32_t KS>
hipError_t launch_rows(const Mxfp4Matmul &p, hipStream_t s) {
  const Args a = args_of(p, kRowsM, kRowsN);
  const uint64_t blocks = tiles_of(a, kRowsM);
  if (blocks * KS * kWave >= kMaxThreads1D) return hipErrorInvalidConfiguration;
  const dim3 grid(static_cast<uint32_t>(blocks)), threads(KS * kWave);
  if (p.out_fp32) hipLaunchKernelGGL((k_mxfp4_rows<KS, true>), grid, threads, 0, s, a);
  else hipLaunchKernelGGL((k_mxfp4_rows<KS, false>), grid, threads, 0, s, a);
  return hipGetLastError();
}

template <uint32_t BM, uint32_t BN, uint32_t WM, uint32_t WN, uint32_t KS = 1>
hipError_t launch_tile(const Mxfp4Matmul &p, hipStream_t s) {
  const Args a = args_of(p, BM, BN);
  const uint64_t blocks = tiles_of(a, BM);
  if (blocks * WM * WN * KS * kWave >= kMaxThreads1D) return hipErrorInvalidConfiguration;
  const dim3 grid(static_cast<uint32_t>(blocks)), threads(WM * WN * KS * kWave);
  if (p.out_fp32) hipLaunchKernelGGL((k_mxfp4_tile<BM, BN, WM, WN, KS, true>), grid, threads, 0, s, a);
  else hipLaunchKernelGGL((k_mxfp4_tile<BM, BN, WM, WN, KS, false>), grid, threads, 0, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mxfp4_matmul(const Mxfp4Matmul &p, hipStream_t s) {
  const bool few = p.mode == kDense ? p.m <= 32 : p.mode == kGroupedRows && p.m <= 32 * static_cast<uint64_t>(p.groups);
  if (few) return p.kblocks >= 16 ? launch_rows<8>(p, s) : launch_rows<2>(p, s);
  auto count = [&](uint64_t edge) {
    const uint64_t rows = (p.m + edge - 1) / edge + (p.mode == kGroupedRows ? p.groups / 2 : 0);
    return rows * ((p.n + edge - 1) / edge) * (p.mode == kGroupedK ? p.groups : 1);
  };
  if (count(128) <= 160) return launch_tile<64, 64, 2, 2, 4>(p, s);
  return launch_tile<128, 128, 2, 2>(p, s);
}

}  // namespace nvfp4
