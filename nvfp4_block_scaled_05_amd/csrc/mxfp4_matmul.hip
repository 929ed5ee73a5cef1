// Products of MXFP4 operands: d = a b^T, a [m][k], b [n][k],
//
//   d[i][j] = sum over blocks B of 32 along k of
//             2^(sa[i][B] - 127) 2^(sb[j][B] - 127) sum_{k in B} a[i][k] b[j][k]
//
// dense, by groups of rows (each group of a's rows has a b of its own) and by
// groups along k (each group of columns gives a d of its own).
//
// v_mfma_scale_f32_16x16x128_f8f6f4 takes the codes as they are in memory and a
// scale byte of each operand for each 32 values. Measured here with FP4
// operands it sums to binary32: sums are exact while the blocks' scales lie
// within 2^6 of each other (products of two codes are multiples of 1/4 up to 36),
// and 3e-8 off in the 2-norm with scales over 2^20, whatever the sum that they
// enter. A zero code counts as 0 under any scale, subnormal results are kept, and
// scale 255 gives NaN. A sum that leaves binary32's range on the way is an
// infinity. So the accumulators are the instruction's own, and d is rounded once
// at the end.
//
// From registers alone, with random operands, the instruction reaches 7.3 PFLOP/s
// on this card: power holds the clock at 1.83 GHz (the 32x32x64 form, which reads
// fewer registers, gets 6.7 at 1.71; zeros 9.4 at 2.34).
#include "codec.h"
#include "launch.h"
#include "matmul.h"

#include <type_traits>

namespace nvfp4 {
namespace {

constexpr uint32_t kBlock = kFp8Block;     // values of a row in one block of scales (a word of four)
constexpr uint32_t kBytes = kBlock / 2;    // bytes of a row in one block
constexpr uint32_t kStepBytes = 128;       // bytes of a row in one step along k: two blocks, a cache line

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

// c + the products of 16x16 rows of 128 values; a lane's scales are bytes SB and SA of sb and sa.
template <uint32_t SB, uint32_t SA>
__device__ __forceinline__ f32x4 product16(u32x4 b, u32x4 a, f32x4 c, uint32_t sb, uint32_t sa) {
  typedef int i32x8 __attribute__((ext_vector_type(8)));
  const i32x8 x = __builtin_bit_cast(i32x8, __builtin_shufflevector(b, b, 0, 1, 2, 3, -1, -1, -1, -1));
  const i32x8 y = __builtin_bit_cast(i32x8, __builtin_shufflevector(a, a, 0, 1, 2, 3, -1, -1, -1, -1));
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, 4, 4, SB, sb, SA, sa);
}
// The same with selectors that fold to constants.
__device__ __forceinline__ f32x4 product16(uint32_t sel_b, uint32_t sel_a, u32x4 b, u32x4 a, f32x4 c, uint32_t sb, uint32_t sa) {
  switch (4 * sel_b + sel_a) {
    case 0: return product16<0, 0>(b, a, c, sb, sa);
    case 1: return product16<0, 1>(b, a, c, sb, sa);
    case 2: return product16<0, 2>(b, a, c, sb, sa);
    case 3: return product16<0, 3>(b, a, c, sb, sa);
    case 4: return product16<1, 0>(b, a, c, sb, sa);
    case 5: return product16<1, 1>(b, a, c, sb, sa);
    case 6: return product16<1, 2>(b, a, c, sb, sa);
    case 7: return product16<1, 3>(b, a, c, sb, sa);
    case 8: return product16<2, 0>(b, a, c, sb, sa);
    case 9: return product16<2, 1>(b, a, c, sb, sa);
    case 10: return product16<2, 2>(b, a, c, sb, sa);
    case 11: return product16<2, 3>(b, a, c, sb, sa);
    case 12: return product16<3, 0>(b, a, c, sb, sa);
    case 13: return product16<3, 1>(b, a, c, sb, sa);
    case 14: return product16<3, 2>(b, a, c, sb, sa);
    default: return product16<3, 3>(b, a, c, sb, sa);
  }
}

template <typename T>
__device__ __forceinline__ T read_lds(uint32_t address) {
  return *reinterpret_cast<__attribute__((address_space(3))) const T *>(static_cast<uintptr_t>(address));
}

// 16 bytes of a row of d from column j on.
template <bool OUT32>
__device__ __forceinline__ void store16(void *d, uint64_t row, uint32_t j, uint32_t n, u32x4 w) {
  constexpr uint32_t per = OUT32 ? 4 : 8;
  if (j + per <= n) {
    if (OUT32) *reinterpret_cast<u32x4_any *>(static_cast<float *>(d) + row + j) = w;
    else *reinterpret_cast<u32x4_any *>(static_cast<uint16_t *>(d) + row + j) = w;
    return;
  }
#pragma unroll
  for (uint32_t e = 0; e < per; ++e) {
    if (j + e >= n) continue;
    if (OUT32) static_cast<uint32_t *>(d)[row + j + e] = w[e];
    else static_cast<uint16_t *>(d)[row + j + e] = static_cast<uint16_t>(e % 2 ? w[e / 2] >> 16 : w[e / 2]);
  }
}

// The rows of 16 lanes each that a wave holds: lane l has columns j + N q .. of row l % 16's (`row`, if `have`), q = l / 16. The
// lanes swap 16-byte pieces first, so that one store writes 64 contiguous bytes of every row: 4096 x 2048 in FP32, 32
// times, takes 420 us so, and 536 with each lane's bytes in four stores.
template <bool OUT32, uint32_t N>
__device__ __forceinline__ void store_rows(void *d, bool have, uint64_t row, uint32_t j, uint32_t n, uint32_t q, const float *v) {
  constexpr uint32_t per = OUT32 ? 4 : 8, kPieces = N / per;
  u32x4 w[kPieces];
#pragma unroll
  for (uint32_t s = 0; s < kPieces; ++s)
#pragma unroll
    for (uint32_t e = 0; e < 4; ++e) w[s][e] = OUT32 ? __float_as_uint(v[s * per + e]) : bf16_pair(v[s * per + 2 * e], v[s * per + 2 * e + 1]);
  auto swap32 = [&](u32x4 &x, u32x4 &y) {  // x's upper 32 lanes and y's lower ones
#pragma unroll
    for (uint32_t e = 0; e < 4; ++e) {
      const auto r = __builtin_amdgcn_permlane32_swap(x[e], y[e], false, false);
      x[e] = r[0], y[e] = r[1];
    }
  };
  auto swap16 = [&](u32x4 &x, u32x4 &y) {  // x's odd 16 lanes and y's even ones
#pragma unroll
    for (uint32_t e = 0; e < 4; ++e) {
      const auto r = __builtin_amdgcn_permlane16_swap(x[e], y[e], false, false);
      x[e] = r[0], y[e] = r[1];
    }
  };
  uint32_t place = q;  // this lane's piece of a store's four
  if constexpr (kPieces == 2) {
    swap32(w[0], w[1]);
    place = q % 2 * 2 + q / 2;
  } else if constexpr (kPieces == 4) {
    swap32(w[0], w[2]);
    swap32(w[1], w[3]);
    swap16(w[0], w[1]);
    swap16(w[2], w[3]);
  }
  if (!have) return;
#pragma unroll
  for (uint32_t s = 0; s < kPieces; ++s) store16<OUT32>(d, row, j + (4 * s + place) * per, n, w[s]);
}

// ---------------------------------------------------------------------------
// Tiles of BM x BN, WM x WN waves, each wave (BM / WM) x (BN / WN) in 16x16
// products. A step along k is two blocks, 128 bytes of every row; two stages
// in LDS, filled by loads straight to LDS. KS times as many waves may share a
// tile, each share with every KS-th step, stages and accumulators of its own,
// which are added up at the end.
//
// Which rows a 16x16 tile takes is free: tile c of four takes rows 4 i + c of
// their 64, i = 0 .. 15 (of two, rows 2 i + c of 32). A lane's rows in the four
// are then neighbours, and their scale words of a block one read of LDS; of each
// word the lane needs the byte of its 32 values, l / 16, and three v_perm gather
// the four bytes to one word, from which the instruction selects.
// The first operand is b, the second a: lane l holds, for row l % 16 of a's
// tile, rows 4 (l / 16) .. + 3 of each of b's four: 16 consecutive columns of d.
//
// LDS layout: rows of 128 bytes, eight 16-byte chunks, chunk g of row r at
// place g ^ (r / 4 % 8) (r / 2 % 8), so that lanes that read one chunk of every fourth
// (second) row meet different banks; the loads to LDS write in lane order, so the permutation
// is in the addresses that they read from. Lane l's fragment of a row and a
// block is chunk l / 16 of four: 32 values, one scale.
//
// A block's products run row tile by row tile. Once a row tile's are issued, the
// next block's fragment is read into the same registers (b's into others, two
// blocks in turn), so every read has almost a block's time. The next step's
// stage is first read in the second block, behind kTurn row tiles, which is
// where everyone meets; the stage that they leave there takes the loads of the
// step after, one or two to a row tile, so that the waves never queue for them.
// ---------------------------------------------------------------------------
template <uint32_t BM, uint32_t BN, uint32_t WM, uint32_t WN, uint32_t KS, bool OUT32>
__global__ __launch_bounds__(WM *WN *KS *kWave) void k_mxfp4_tile(Args p) {
  constexpr uint32_t kWaves = WM * WN;
  constexpr uint32_t TM = BM / WM, TN = BN / WN, MI = TM / 16, NI = TN / 16;
  constexpr uint32_t CA = MI < 4 ? MI : 4, CB = NI < 4 ? NI : 4;  // tiles that share their rows
  constexpr uint32_t kLoadA = BM / 8 / kWaves, kLoadB = BN / 8 / kWaves;  // loads of 8 rows that a wave makes
  constexpr uint32_t kGroups = (BM + BN) / 64 * 2, kLoadS = (kGroups + kWaves - 1) / kWaves;  // loads of 64 scale words
  constexpr uint32_t kLoads = kLoadA + kLoadB + kLoadS;
  constexpr uint32_t kTurn = MI > 4 ? 2 : 1;
  constexpr uint32_t kPer = (kLoads + 2 * MI - kTurn - 2) / (2 * MI - kTurn - 1);  // loads to a row tile
  constexpr uint32_t kFirst = (MI - kTurn) * kPer;                                 // those of the second block
  constexpr uint32_t kStage = (BM + BN) * kStepBytes, kBlockScales = (BM + BN) * 4, kStageScales = 2 * kBlockScales;
  static_assert(MI % CA == 0 && NI % CB == 0 && CA != 3 && CB != 3, "tiles in fours or a pair");
  static_assert(BM % (8 * kWaves) == 0 && BN % (8 * kWaves) == 0 && BM % 64 == 0 && BN % 64 == 0, "loads of whole rows");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[KS][2 * kStage];
  __shared__ __attribute__((aligned(1024))) uint8_t scales[KS][2 * kStageScales];

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
  // (these are the same in all lanes, which the compiler does not see)
  const uint32_t kb_first = __builtin_amdgcn_readfirstlane(part.kb0), kb_end = __builtin_amdgcn_readfirstlane(part.zero ? part.kb0 : part.kb_end);
  const uint32_t m0 = __builtin_amdgcn_readfirstlane(part.m0), n0 = tn * BN;
  const uint32_t rows_a = __builtin_amdgcn_readfirstlane(part.m_end) - m0, rows_b = p.n - n0;  // from the tile's first on
  const uint32_t pitch = p.kblocks * kBytes;  // at most 2^22
  const uint8_t *a = p.a + static_cast<uint64_t>(m0) * pitch, *b = p.b + static_cast<uint64_t>(n0) * pitch;
  const uint32_t *sa = p.sa + m0, *sb = p.sb + n0;
  if (p.mode == kGroupedRows) {
    const uint64_t group = __builtin_amdgcn_readfirstlane(part.group);
    b += group * p.n * pitch;
    sb += group * p.n * p.kblocks;
  }

  // Loads of a step: the two blocks from kb on, which are inside the rows. (The last step of an odd number of blocks
  // begins a block earlier, and its first block is not used again; of rows of one block the second is the first again.)
  const uint32_t lds_data = lds_address(&lds[share][0]), lds_scales = lds_address(&scales[share][0]);
  const uint32_t last_start = p.kblocks < 2 ? 0 : p.kblocks - 2, chunk_bits = p.kblocks < 2 ? 3 : 7;
  const uint32_t r8 = lane / 8, chunk0_a = (lane % 8 ^ r8 / CA) << 4 & chunk_bits << 4, chunk0_b = (lane % 8 ^ r8 / CB) << 4 & chunk_bits << 4;
  const uint32_t groups_a = (rows_a + 7) / 8, groups_b = (rows_b + 7) / 8;
  const uint32_t from_row = r8 * pitch;  // in eight rows; of the last eight that there are:
  const uint32_t from_last_a = min(r8, rows_a - 1 - (groups_a - 1) * 8) * pitch, from_last_b = min(r8, rows_b - 1 - (groups_b - 1) * 8) * pitch;
  auto load = [&](uint32_t i, uint32_t kb, uint32_t stage) {
    const uint32_t start = min(kb, last_start);
    if (i < kLoadA + kLoadB) {
      const bool of_a = i < kLoadA;
      const uint32_t at = of_a ? wave * kLoadA + i : wave * kLoadB + i - kLoadA;  // eights of the tile's rows
      const uint32_t last = (of_a ? groups_a : groups_b) - 1, group = min(at, last);  // those past the end repeat the last ones
      const uint32_t from = group == last ? (of_a ? from_last_a : from_last_b) : from_row;
      load16_to_lds(lds_data + stage * kStage + (of_a ? 0 : BM * kStepBytes) + at * 1024, (of_a ? a : b) + static_cast<uint64_t>(start) * kBytes + group * 8 * pitch,
                    ((of_a ? chunk0_a : chunk0_b) ^ (8 / (of_a ? CA : CB) * at & chunk_bits) << 4) + from);
    } else {
      const uint32_t any = __builtin_amdgcn_readfirstlane((wave * kLoadS + i - kLoadA - kLoadB) % kGroups), w = any % (kGroups / 2);
      const uint64_t at = min(start + any / (kGroups / 2), p.kblocks - 1);
      const bool of_a = w < BM / 64;
      const uint32_t r = (of_a ? w : w - BM / 64) * 64 + lane;
      load4_to_lds(lds_scales + stage * kStageScales + any * 256, of_a ? sa + at * p.m : sb + at * p.n, 4 * min(r, (of_a ? rows_a : rows_b) - 1));
    }
  };

  const uint32_t wm = wave % WM, wn = wave / WM;
  const uint32_t i16 = lane % 16, q = lane / 16;
  f32x4 acc[MI][NI];
#pragma unroll
  for (uint32_t i = 0; i < MI; ++i)
#pragma unroll
    for (uint32_t j = 0; j < NI; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  // Where this lane reads in a stage: its rows' first blocks (the second ones are 64 bytes on or back) and scales; the
  // other tiles' are at fixed distances.
  u32x4 va[MI], vb[2][NI];
  uint32_t fa[MI / CA], fb[2][NI / CB];
  const uint32_t row_a = wm * TM + CA * i16, row_b = wn * TN + CB * i16;
  uint32_t at_a[2], at_b[2], at_sa = lds_scales + 4 * row_a, at_sb = lds_scales + 4 * (BM + row_b);
  at_a[0] = lds_data + row_a * kStepBytes + ((q ^ (row_a / CA & 7)) << 4);
  at_b[0] = lds_data + (BM + row_b) * kStepBytes + ((q ^ (row_b / CB & 7)) << 4);
  at_a[1] = at_a[0] ^ 64;
  at_b[1] = at_b[0] ^ 64;
  uint32_t to_other = kStage, to_other_scales = kStageScales;  // the distance to the other stage, and back
  auto other_stage = [&] {
    at_a[0] += to_other, at_a[1] += to_other, at_b[0] += to_other, at_b[1] += to_other;
    at_sa += to_other_scales, at_sb += to_other_scales;
    to_other = -to_other, to_other_scales = -to_other_scales;
  };
  // v_perm's selectors: byte q of two words side by side
  const uint32_t pick = 0x0C0C0400u + q * 0x0101u, side_by_side = 0x05040100u;
  auto scale_bytes = [&](uint32_t at, auto tiles) {
    if constexpr (decltype(tiles)::value == 4) {
      const u32x4 w = read_lds<u32x4>(at);
      return __builtin_amdgcn_perm(__builtin_amdgcn_perm(w[3], w[2], pick), __builtin_amdgcn_perm(w[1], w[0], pick), side_by_side);
    } else {
      typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
      const u32x2 w = read_lds<u32x2>(at);
      return __builtin_amdgcn_perm(w[1], w[0], pick);
    }
  };
  auto read_a = [&](uint32_t half, uint32_t i) {
    va[i] = read_lds<u32x4>(at_a[half] + (i / CA * 16 * CA + i % CA) * kStepBytes);
  };
  auto read_b = [&](uint32_t half, uint32_t j) {
    vb[half][j] = read_lds<u32x4>(at_b[half] + (j / CB * 16 * CB + j % CB) * kStepBytes);
    if (j % CB == 0) fb[half][j / CB] = scale_bytes(at_sb + half * kBlockScales + j / CB * 64 * CB, std::integral_constant<uint32_t, CB>{});
  };
  auto read_scales_a = [&](uint32_t half, uint32_t g) { fa[g] = scale_bytes(at_sa + half * kBlockScales + g * 64 * CA, std::integral_constant<uint32_t, CA>{}); };
  auto products = [&](uint32_t half, uint32_t i) {
#pragma unroll
    for (uint32_t j = 0; j < NI; ++j) acc[i][j] = product16(j % CB, i % CA, vb[half][j], va[i], acc[i][j], fb[half][j / CB], fa[i / CA]);
#pragma unroll
    for (uint32_t j = 0; j < NI; ++j) asm volatile("" : "+v"(acc[i][j]));  // (they stay here: the compiler moves them behind the barrier)
  };

  if (kb_first < kb_end) {
    // (a share without a step in the last round loads something and leaves it)
#pragma unroll
    for (uint32_t i = 0; i < kLoads; ++i) load(i, kb_first + 2 * share, 0);
    wait_loads();
    lds_barrier();
    if (kb_first + 2 * KS < kb_end) {
#pragma unroll
      for (uint32_t i = 0; i < kFirst && i < kLoads; ++i) load(i, kb_first + 2 * KS + 2 * share, 1);
    }
#pragma unroll
    for (uint32_t j = 0; j < NI; ++j) read_b(0, j);
#pragma unroll
    for (uint32_t i = 0; i < MI; ++i) {
      read_a(0, i);
      if (i % CA == 0) read_scales_a(0, i / CA);
    }
    uint32_t stage = 0, first = kb_first;
    for (; first + 2 * share + 1 < kb_end; first += 2 * KS, stage ^= 1) {  // (all but the last round are whole for every share)
      // Past the last round nothing is loaded, no one waits, and what is read is not used.
#pragma unroll
      for (uint32_t i = 0; i < MI; ++i) {
        products(0, i);
        read_a(1, i);
        if (i % CA == CA - 1) read_scales_a(1, i / CA);
#pragma unroll
        for (uint32_t j = i * NI / MI; j < (i + 1) * NI / MI; ++j) read_b(1, j);
        if (kFirst + i * kPer < kLoads && first + 2 * KS < kb_end) {
#pragma unroll
          for (uint32_t k = kFirst + i * kPer; k < kFirst + (i + 1) * kPer && k < kLoads; ++k) load(k, first + 2 * KS + 2 * share, stage ^ 1);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (uint32_t i = 0; i < MI; ++i) {
        products(1, i);
        if (i + 1 == kTurn) {
          if (first + 2 * KS < kb_end) {
            wait_loads();   // the next step's loads are in,
            lds_barrier();  // everyone's are, and everyone has read this stage
          }
          other_stage();
#pragma unroll
          for (uint32_t k = 0; k < kTurn; ++k) read_a(0, k);
        } else if (i >= kTurn) {
          read_a(0, i);
        }
        if (i % CA == CA - 1) read_scales_a(0, i / CA);
        if (i + 1 >= kTurn) {
          constexpr uint32_t slots = MI - kTurn + 1;
#pragma unroll
          for (uint32_t j = (i + 1 - kTurn) * NI / slots; j < (i + 2 - kTurn) * NI / slots; ++j) read_b(0, j);
        }
        if (i >= kTurn && first + 4 * KS < kb_end) {
#pragma unroll
          for (uint32_t k = (i - kTurn) * kPer; k < (i + 1 - kTurn) * kPer && k < kLoads; ++k) load(k, first + 4 * KS + 2 * share, stage);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if (first + 2 * share + 1 == kb_end) {  // a last step of one block
      if (first + 2 * share > last_start) {   // which is the second of its stage
#pragma unroll
        for (uint32_t j = 0; j < NI; ++j) {
          vb[0][j] = read_lds<u32x4>(at_b[1] + (j / CB * 16 * CB + j % CB) * kStepBytes);
          if (j % CB == 0) fb[0][j / CB] = scale_bytes(at_sb + kBlockScales + j / CB * 64 * CB, std::integral_constant<uint32_t, CB>{});
        }
#pragma unroll
        for (uint32_t i = 0; i < MI; ++i) {
          read_a(1, i);
          if (i % CA == 0) read_scales_a(1, i / CA);
        }
      }
#pragma unroll
      for (uint32_t i = 0; i < MI; ++i) products(0, i);
    }
  }

  if (KS > 1) {  // the shares' sums meet in the first one's registers, in their order
    f32x4(*sums)[MI * NI][kWaves][kWave] = reinterpret_cast<f32x4(*)[MI * NI][kWaves][kWave]>(&lds[0][0]);
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
    const uint32_t r = wm * TM + i / CA * 16 * CA + CA * i16 + i % CA;
    const uint64_t row = d_base + static_cast<uint64_t>(m0 + r) * p.n;
#pragma unroll
    for (uint32_t g = 0; g < NI / CB; ++g) {
      float v[4 * CB];
#pragma unroll
      for (uint32_t e = 0; e < 4 * CB; ++e) v[e] = acc[i][CB * g + e % CB][e / CB];
      store_rows<OUT32, 4 * CB>(p.d, r < rows_a, row, n0 + wn * TN + 16 * CB * g, p.n, q, v);
    }
  }
}

// ---------------------------------------------------------------------------
// Few rows: all of a's and kRowsN of b's to a workgroup, the pairs of blocks along k
// dealt out to its KS waves, each with accumulators of its own, which meet in LDS
// at the end, in the order of the waves. Operands go from memory to registers: each
// row of b is read once and by one wave, so LDS would only add a step. U pairs of
// blocks make a round, which ends at the first block past the end; that is a branch
// before each block's products, and the compiler loads a block's operands behind
// it, so blocks come one after the other (40 registers with U 4, not the 96 that
// all of a round's would take), and it is the eight waves of a workgroup that
// overlap. Bound by that: 16 x 8192 x 5120 takes 5.7 us with its weights in the
// Infinity Cache and 9.3 from HBM, where they are 4.4 at a copy's rate. Lane l's 16
// bytes of a block are block l / 16 of four of row l % 16.
// ---------------------------------------------------------------------------
constexpr uint32_t kRowsM = 32, kRowsN = 32;

template <uint32_t KS, uint32_t MT, uint32_t U, bool OUT32>
__global__ __launch_bounds__(KS *kWave) void k_mxfp4_rows(Args p) {
  static_assert(16 * MT <= kRowsM, "rows");
  __shared__ f32x4 red[KS][MT * 2][kWave];
  const uint32_t n0 = blockIdx.x * kRowsN;
  const uint32_t lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const uint32_t i16 = lane % 16, q = lane / 16;
  const uint64_t pitch = static_cast<uint64_t>(p.kblocks) * kBytes;
  // tile t of b takes rows 8 (i / 4) + 4 t + i % 4, so that a lane ends with 8 consecutive columns of d
  uint32_t row_a[MT], row_b[2];
  const uint8_t *a[MT], *b[2];
#pragma unroll
  for (uint32_t i = 0; i < MT; ++i) {
    row_a[i] = min(16 * i + i16, p.m - 1);
    a[i] = p.a + row_a[i] * pitch + 16 * q;
  }
#pragma unroll
  for (uint32_t t = 0; t < 2; ++t) {
    row_b[t] = min(n0 + 8 * (i16 / 4) + 4 * t + i16 % 4, p.n - 1);
    b[t] = p.b + row_b[t] * pitch + 16 * q;
  }

  f32x4 acc[MT][2];
#pragma unroll
  for (uint32_t i = 0; i < MT; ++i) acc[i][0] = acc[i][1] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  for (uint32_t kb0 = 2 * wave; kb0 < p.kblocks; kb0 += 2 * U * KS) {
    u32x4 wa[2 * U][MT], wb[2 * U][2];
    uint32_t fa[2 * U][MT], fb[2 * U][2];
#pragma unroll
    for (uint32_t u = 0; u < 2 * U; ++u) {
      const uint64_t kb = min(kb0 + u / 2 * 2 * KS + u % 2, p.kblocks - 1);  // past the end: loaded again, not used
#pragma unroll
      for (uint32_t t = 0; t < 2; ++t) {
        wb[u][t] = *reinterpret_cast<const u32x4 *>(b[t] + kb * kBytes);
        fb[u][t] = p.sb[kb * p.n + row_b[t]];
      }
#pragma unroll
      for (uint32_t i = 0; i < MT; ++i) {
        wa[u][i] = *reinterpret_cast<const u32x4 *>(a[i] + kb * kBytes);
        fa[u][i] = p.sa[kb * p.m + row_a[i]];
      }
    }
#pragma unroll
    for (uint32_t u = 0; u < 2 * U; ++u) {
      if (kb0 + u / 2 * 2 * KS + u % 2 >= p.kblocks) break;
#pragma unroll
      for (uint32_t i = 0; i < MT; ++i)
#pragma unroll
        for (uint32_t t = 0; t < 2; ++t) acc[i][t] = product16<0, 0>(wb[u][t], wa[u][i], acc[i][t], fb[u][t] >> (8 * q), fa[u][i] >> (8 * q));
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
    const uint32_t m = 16 * (it / 2) + i16;
    if (m < p.m) store4<OUT32>(p.d, static_cast<uint64_t>(m) * p.n, n0 + 8 * q + 4 * (it % 2), p.n, v);
  }
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

template <uint32_t KS, uint32_t MT, uint32_t U>
hipError_t launch_rows(const Mxfp4Matmul &p, hipStream_t s) {
  const Args a = args_of(p, kRowsM, kRowsN);
  const dim3 grid(a.tiles_n), threads(KS * kWave);
  if (p.out_fp32) hipLaunchKernelGGL((k_mxfp4_rows<KS, MT, U, true>), grid, threads, 0, s, a);
  else hipLaunchKernelGGL((k_mxfp4_rows<KS, MT, U, false>), grid, threads, 0, s, a);
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

// Which kernel. Times in us, of one session, the kernel alone.
//   Few rows, dense, and columns for at most a workgroup of 64x64 tiles a CU, against the tiles below:
//     1 x 8192 x 5120     5.1 / 8.2      32 x 8192 x 5120  7.2 / 8.3     32 x 2048 x 2048  4.3 / 5.6
//     but 64 x 8192 x 5120  10.2 / 8.5;  16 x 28672 x 8192  31 / 23
//   Groups of up to 64 rows on average, by the buffer's rows: 64 rows high, against 128x128 tiles
//   and a kernel of few rows by groups:
//     64 groups, 1472 rows x 4096 x 2048  51 / 63 / 78      32 groups, 992 rows  27 / 28 / 37
//     64 groups, 4096 rows x 4096 x 2048  63 / 71 / 132
//   Up to one tile a CU the waves share the blocks along k, in the smallest tiles for which that holds:
//   64x64 by four, 64x128 by two, 128x128 by two, against each other and the same without shares
//     128 x 8192 x 5120   9.3 / 13.9 / 15.1, 10.6     256 x 4096 x 4096   8.0 / 11.5 / 12.5, 8.8
//     512 x 4096 x 4096  14.6 / 10.9 / 14.3, 12.6    1280 x 2048 x 4096  22.3 / 20.4 / 13.9, 17.1
//     2048 x 2048 x 2048  20 / 13.3 / 10.2, 10.8
//   256x256 tiles where their rounds over 256 CUs, taken as 3, are no longer than those of 128x128 tiles
//   over 512 places, taken as 2:
//     4096 x 4096 x 4096  39 / 47       8192 x 8192 x 5120  172 / 229      3000 x 8192 x 5120  82 / 83
//     64 groups, 73600 rows x 4096 x 2048  470 / 571      32 weight gradients of 4096 x 2048  420 / 530
//     but 2048 x 4096 x 4096, which takes 128x128, 33 / 26
hipError_t launch_mxfp4_matmul(const Mxfp4Matmul &p, hipStream_t s) {
  // by groups of rows, every second group's last tile is taken to be a partial one
  auto count = [&](uint64_t bm, uint64_t bn) {
    const uint64_t rows = (p.m + bm - 1) / bm + (p.mode == kGroupedRows ? p.groups / 2 : 0);
    return rows * ((p.n + bn - 1) / bn) * (p.mode == kGroupedK ? p.groups : 1);
  };
  if (p.mode == kGroupedRows) {
    if (p.m <= 64 * static_cast<uint64_t>(p.groups)) return launch_tile<64, 128, 2, 2>(p, s);
  } else {
    if (p.mode == kDense && p.m <= kRowsM && count(64, 64) <= 256) {
      // (a wave's share is best at least a round's pairs of blocks)
      if (p.m <= 16) return p.kblocks >= 16 ? launch_rows<8, 1, 4>(p, s) : launch_rows<2, 1, 4>(p, s);
      return p.kblocks >= 16 ? launch_rows<8, 2, 2>(p, s) : launch_rows<2, 2, 2>(p, s);
    }
    if (count(64, 64) <= 256) return launch_tile<64, 64, 2, 2, 4>(p, s);
    if (count(64, 128) <= 256) return launch_tile<64, 128, 2, 2, 2>(p, s);
    if (count(128, 128) <= 256) return launch_tile<128, 128, 2, 2, 2>(p, s);
  }
  if (3 * ((count(256, 256) + 255) / 256) <= 2 * ((count(128, 128) + 511) / 512)) return launch_tile<256, 256, 2, 4>(p, s);
  return launch_tile<128, 128, 2, 2>(p, s);
}

}  // namespace nvfp4
