// Products of block-scaled FP8 operands: d = a b^T, a [m][k], b [n][k],
//
//   d[i][j] = sum over blocks B of 128 along k of
//             sa[B][i] * sb[B][j or j / 128] * sum_{k in B} a[i][k] b[j][k]
//
// dense, by groups of rows (each group of a's rows has a b of its own) and by
// groups along k (each group of columns gives a d of its own).
//
// The matrix cores' FP8 forms do not sum in binary32: measured here, they
// line up each eight products with the largest of them and drop what lies
// more than 13 bits below it, which puts a sum of 128 up to 1.4e-4 of its
// terms' magnitudes off (4.6e-5 of the result in the 2-norm). The BF16 form
// is exact to binary32 (2e-7, 4e-8). So the codes stay FP8 in memory and in
// LDS, are widened in registers (E4M3 values are BF16 values; one
// instruction makes two, beside the matrix core's work), and four
// v_mfma_f32_16x16x32_bf16 sum a block's products of a 16x16 tile. The sum
// then enters the accumulators, binary32 as well, by one fused multiply-add
// with the product of the block's two scales; d is rounded once at the end.
//
// That product may leave binary32's range where the term does not (1e-25 * 1e-25 *
// 2e7), or where the sum is 0. (b in 1x128 blocks: the sum times a's scale enters by
// a multiply-add with b's, and that first product may.) The tile kernels therefore
// look at the scales that they use (near()), and where that could be, the wave
// computes its part of the tile again, by add_far(), which multiplies mantissas and
// adds exponents. Looking costs 1% in 256x256 tiles with 128x128 blocks of b (8192 x
// 8192 x 5120 498 -> 503 us) and 2 to 5% elsewhere (512 x 4096 x 4096 22.1 -> 22.7, 32
// weight gradients of 4096 x 2048 664 -> 680); a product whose every tile is computed
// again takes ten times as long. The few-row kernel, which has time beside its loads,
// always takes add_far().
#include "codec.h"
#include "launch.h"

namespace nvfp4 {
namespace {

constexpr uint32_t kWave = 64;
constexpr uint32_t kBlock = kFp8Block;  // bytes of a row in one step along k

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));  // rows of d start at any element

struct Args {
  const uint8_t *a, *b;
  const float *sa, *sb;
  void *d;
  uint32_t m, n, kblocks;
  uint32_t sa_stride, sb_stride;
  uint32_t mode;
  const int32_t *offsets;
  uint32_t groups;
  uint32_t tiles_m, tiles_n;  // of the grid (by groups along k: of one group)
};

// The part of the product that a tile of BM rows works on.
struct Part {
  uint32_t m0, m_end;    // rows of a and d: m0 .. m_end - 1
  uint32_t kb0, kb_end;  // blocks along k
  uint32_t group;
  bool zero;             // rows past the last group: d is cleared
};

__device__ __forceinline__ uint32_t clamped(int32_t v, uint32_t most) {
  return v < 0 ? 0u : min(static_cast<uint32_t>(v), most);
}

// Tile `tile` of the row tiles of all groups, then of the rows past the last
// group. Every wave looks it up by itself: lane l takes groups 4 l .. 4 l + 3.
// Offsets are clamped to the rows there are, so any contents stay in bounds.
template <uint32_t BM>
__device__ __forceinline__ Part find_rows(const Args &p, uint32_t tile) {
  const uint32_t lane = threadIdx.x % kWave;
  uint32_t start[5], tiles[4], sum = 0;
#pragma unroll
  for (uint32_t i = 0; i < 5; ++i) start[i] = clamped(p.offsets[min(4 * lane + i, p.groups)], p.m);
#pragma unroll
  for (uint32_t i = 0; i < 4; ++i) {
    tiles[i] = start[i + 1] > start[i] ? (start[i + 1] - start[i] + BM - 1) / BM : 0;
    sum += tiles[i];
  }
  uint32_t scan = sum;
#pragma unroll
  for (uint32_t d = 1; d < kWave; d *= 2) {
    const uint32_t up = __shfl_up(scan, d);
    scan += lane >= d ? up : 0u;
  }
  const uint64_t past = __ballot(scan > tile);
  Part r{0, 0, 0, p.kblocks, 0, false};
  if (past == 0) {
    const uint32_t total = __builtin_amdgcn_readlane(scan, kWave - 1);
    const uint64_t m0 = clamped(p.offsets[p.groups], p.m) + static_cast<uint64_t>(tile - total) * BM;
    r.m0 = static_cast<uint32_t>(min(m0, static_cast<uint64_t>(p.m)));
    r.m_end = p.m;
    r.zero = true;
    return r;
  }
  const uint32_t l = __builtin_ctzll(past);
  uint32_t rest = tile - (__builtin_amdgcn_readlane(scan, l) - __builtin_amdgcn_readlane(sum, l));
#pragma unroll
  for (uint32_t i = 0; i < 4; ++i) {
    const uint32_t n = __builtin_amdgcn_readlane(tiles[i], l);
    if (rest < n) {
      r.m0 = __builtin_amdgcn_readlane(start[i], l) + rest * BM;
      r.m_end = __builtin_amdgcn_readlane(start[i + 1], l);
      r.group = 4 * l + i;
      break;
    }
    rest -= n;
  }
  return r;
}

// Workgroup `id`'s tile. Workgroups go to the eight XCDs in turn, each of
// which has an L2 of its own: so each XCD gets runs of 32 consecutive places,
// and places run through patches of kPatch tile rows, column by column, so
// that the 32 tiles that an XCD works on at a time share their operands.
constexpr uint32_t kXcds = 8, kRun = 32, kPatch = 4;
__device__ __forceinline__ void tile_of(uint32_t id, const Args &p, uint32_t &tm, uint32_t &tn) {
  const uint32_t total = gridDim.x;
  if (id < total / (kXcds * kRun) * (kXcds * kRun)) {
    const uint32_t in = id % (kXcds * kRun);
    id = id - in + in % kXcds * kRun + in / kXcds;
  }
  const uint32_t rows = total / p.tiles_n, band = id / (kPatch * p.tiles_n), in = id - band * kPatch * p.tiles_n;
  const uint32_t high = min(kPatch, rows - band * kPatch);
  tm = band * kPatch + in % high;
  tn = in / high;
}

template <bool OUT32>
__device__ __forceinline__ void store1(void *d, uint64_t at, float v) {
  if (OUT32) static_cast<float *>(d)[at] = v;
  else static_cast<uint16_t *>(d)[at] = static_cast<uint16_t>(bf16_pair(v, 0.0f));
}

// Values v[0 .. N - 1] to columns j .. j + N - 1 of a row of d that starts at `row`.
template <bool OUT32, uint32_t N>
__device__ __forceinline__ void store(void *d, uint64_t row, uint32_t j, uint32_t n, const float *v) {
  constexpr uint32_t per = OUT32 ? 4 : 8;
#pragma unroll
  for (uint32_t i = 0; i < N; i += per) {
    if (j + i + per <= n) {
      u32x4_any w;
#pragma unroll
      for (uint32_t q = 0; q < 4; ++q) w[q] = OUT32 ? __float_as_uint(v[i + q]) : bf16_pair(v[i + 2 * q], v[i + 2 * q + 1]);
      if (OUT32) *reinterpret_cast<u32x4_any *>(static_cast<float *>(d) + row + j + i) = w;
      else *reinterpret_cast<u32x4_any *>(static_cast<uint16_t *>(d) + row + j + i) = w;
    } else {
#pragma unroll
      for (uint32_t q = 0; q < per; ++q)
        if (j + i + q < n) store1<OUT32>(d, row + j + i + q, v[i + q]);
    }
  }
}

template <bool OUT32>
__device__ __forceinline__ void store4(void *d, uint64_t row, uint32_t j, uint32_t n, f32x4 v) {
  if (j + 4 <= n) {
    if (OUT32) {
      *reinterpret_cast<u32x4_any *>(static_cast<float *>(d) + row + j) =
          u32x4_any{__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3])};
    } else {
      typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));
      *reinterpret_cast<u32x2_any *>(static_cast<uint16_t *>(d) + row + j) = u32x2_any{bf16_pair(v[0], v[1]), bf16_pair(v[2], v[3])};
    }
  } else {
#pragma unroll
    for (uint32_t q = 0; q < 4; ++q)
      if (j + q < n) store1<OUT32>(d, row + j + q, v[q]);
  }
}

// Loads straight to LDS, 16 bytes or 4 a lane: lane l's go to `to` + 16 l (4 l),
// from `from` + `offset`. Written out, since the compiler waits for every
// such load before the next LDS read, whichever stage it reads. They have no
// destination register; wait_loads() waits for all of them.
__device__ __forceinline__ uint32_t lds_address(const void *p) {
  return static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const void *)p));
}
// m0 holds the LDS address and is put back; it needs one wait state before the load.
__device__ __forceinline__ void load16_to_lds(uint32_t to, const void *from, uint32_t offset) {
  uint32_t keep;
  asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %2, %3\n\ts_mov_b32 m0, %0"
               : "=&s"(keep) : "s"(to), "v"(offset), "s"(from) : "memory");
}
__device__ __forceinline__ void load4_to_lds(uint32_t to, const void *from, uint32_t offset) {
  uint32_t keep;
  asm volatile("s_mov_b32 %0, m0\n\ts_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %2, %3\n\ts_mov_b32 m0, %0"
               : "=&s"(keep) : "s"(to), "v"(offset), "s"(from) : "memory");
}
__device__ __forceinline__ void wait_loads() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// 16 codes to BF16: the eight of the first two words and of the last two.
struct Wide {
  bf16x8 lo, hi;
};
__device__ __forceinline__ bf16x8 widen8(uint32_t x, uint32_t y) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x, 1.0f, false), b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x, 1.0f, true);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(y, 1.0f, false), d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(y, 1.0f, true);
  return bf16x8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}
__device__ __forceinline__ Wide widen(u32x4 w) { return Wide{widen8(w.x, w.y), widen8(w.z, w.w)}; }

// A block's sums of 128 products of a 16x16 tile.
__device__ __forceinline__ f32x4 block_sum(const Wide &b0, const Wide &b1, const Wide &a0, const Wide &a1) {
  f32x4 c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b0.lo, a0.lo, f32x4{0.0f, 0.0f, 0.0f, 0.0f}, 0, 0, 0);
  c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b0.hi, a0.hi, c, 0, 0, 0);
  c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(b1.lo, a1.lo, c, 0, 0, 0);
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(b1.hi, a1.hi, c, 0, 0, 0);
}

// Whether a block's sum can be scaled the short way: with 128x128 blocks of b,
// where sa * sb is 0 for a 0 scale or a normal number; with 1x128 blocks, where
// c * sa is, for any sum c other than 0: 2^-18 to 2^24.7.
template <bool SBV>
__device__ __forceinline__ bool near(float sa, float sb) {
  constexpr int kNormal = 0x108;  // of either sign
  if (!SBV) return __builtin_amdgcn_classf(sa * sb, kNormal) || sa == 0.0f || sb == 0.0f;
  return fabsf(sa) < 0x1p103f && (fabsf(sa) >= 0x1p-108f || sa == 0.0f);
}

// acc + c * sa * sb for scales of any size: the term is what binary32 holds of it,
// an infinity only where it is too large.
__device__ __forceinline__ f32x4 add_far(f32x4 acc, f32x4 c, float sa, f32x4 sb) {
  const float ma = __builtin_amdgcn_frexp_mantf(sa);
  const int ea = __builtin_amdgcn_frexp_expf(sa);
#pragma unroll
  for (uint32_t e = 0; e < 4; ++e)
    acc[e] += __builtin_amdgcn_ldexpf(c[e] * (ma * __builtin_amdgcn_frexp_mantf(sb[e])), ea + __builtin_amdgcn_frexp_expf(sb[e]));
  return acc;
}

// ---------------------------------------------------------------------------
// Tiles of BM x BN, WM x WN waves, each wave (BM / WM) x (BN / WN). A step
// along k is one block of 128 bytes of every row; two stages in LDS, the next
// one filled by loads straight to LDS while the matrix cores work on this one.
// KS times as many waves may share a tile, each share with every KS-th block,
// stages and accumulators of its own, which are added up at the end.
//
// At 8192 x 8192 x 5120 this takes 580 to 607 us (1.15 PFLOP/s, by the box) in
// 128x128 tiles, two workgroups a CU. The widening and the scaling are 3 vector
// instructions for each v_mfma; measured alone, a v_mfma takes 17 cycles with up
// to two of them beside it and 22 with three, and the mix of this kernel from
// registers only 25, against 29 here. The rest is power: the clock drops to
// 2.1 GHz. 32x32x16 v_mfma, which leave more room beside them, need 5% fewer
// cycles and take 590 us, at 1.9 GHz.
//
// PHASED: 256x256 tiles, waves of 128x64, which widen and read LDS less (2.5
// vector instructions a v_mfma), but one workgroup a CU, whose waves would all
// wait, then read and widen b, and leave the matrix cores idle together: 570
// us. So the two waves of each SIMD run half a step apart. Waves 0 .. 3 (upper
// half of the rows) begin a step at one barrier and pass the next one in the
// middle of it, where waves 4 .. 7 begin theirs: 535 to 545 us, and 484 to 516 us
// (1.33 to 1.42 PFLOP/s) with the instructions in groups, below.
// What that needs of the two stages: each half of the waves loads its own rows
// of a, at its own steps' beginnings; b is read at a step's beginning only, so
// the stage that the lower half has read by the middle of its step k, which is
// where the upper half begins step k + 1, takes b of step k + 2 then, loaded by
// the upper half. Each load has a whole step's time.
//
// LDS layout: rows of 128 bytes, eight 16-byte chunks, chunk g of row r at
// place g ^ f(r), so that lanes that read one chunk of neighbouring rows meet
// different banks; the loads to LDS write in lane order, so the permutation
// is in the addresses that they read from.
// The matrix core's first operand is b, its second a: lane l then holds, for
// row l % 16 of a, four consecutive rows 4 (l / 16) .. of the 16x16 tile's
// b. Which rows of b a tile takes is free: tile j of G takes rows 4 G q + 4 j
// + r of a group of 16 G as its rows 4 q + r, so that a lane ends with 4 G
// consecutive columns of d: 16 bytes, which four lanes continue to 64. (With
// G 4 a store is 16 bytes of every 64; the FP32 weight gradients of 32 groups,
// 4096 x 2048 each, took 780 us so, and took 711 in the same tiles without.)
// ---------------------------------------------------------------------------
// f(r) of b: with that order of its rows, eight lanes that follow each other get eight values
template <uint32_t G>
__device__ __forceinline__ uint32_t swizzle_b(uint32_t r) { return (r & 3) | (r / (4 * G) & 1) << 2; }

template <uint32_t BM, uint32_t BN, uint32_t WM, uint32_t WN, uint32_t KS, bool PHASED, bool SBV, bool OUT32>
__global__ __launch_bounds__(WM *WN *KS *kWave) void k_fp8_tile(Args p) {
  constexpr uint32_t kWaves = WM * WN;
  constexpr uint32_t TM = BM / WM, TN = BN / WN, MI = TM / 16, NI = TN / 16;
  constexpr uint32_t G = OUT32 ? 1 : 2, NG = NI / G;  // 16-row tiles of b that share 16 G rows
  constexpr uint32_t kLoadA = BM / 8 / kWaves, kLoadB = BN / 8 / kWaves;  // loads of 8 rows that a wave makes
  constexpr uint32_t kGroups = (BM + BN) / 64, kLoadS = (kGroups + kWaves - 1) / kWaves;
  static_assert((NI == 2 || NI == 4) && BM % (8 * kWaves) == 0 && BN % (8 * kWaves) == 0, "tile shape");
  // In groups of instructions (below) where the registers hold that.
  constexpr bool kGrouped = NI == 4 && MI >= 4 && !(PHASED && SBV);
  constexpr uint32_t kTurn = kGrouped ? 2 : 3;  // of a phased wave's 8 row tiles, those before the barrier; one more or less: 1 to 4% slower
  static_assert(!PHASED || (BM == 256 && BN == 256 && WM == 2 && WN == 4 && KS == 1), "phased shape");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[KS][2][(BM + BN) * kBlock];
  __shared__ __attribute__((aligned(16))) float scales[KS][2][BM + BN];
  __shared__ bool far_waves[KS > 1 ? kWaves : 1];  // of the first share's waves, those whose other shares met scales that are not near

  const uint32_t lane = threadIdx.x % kWave, any_wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const uint32_t wave = any_wave % kWaves, share = any_wave / kWaves;  // of the waves that share a tile's blocks along k
  uint32_t tm, tn;
  tile_of(blockIdx.x, p, tm, tn);
  Part part{tm * BM, p.m, 0, p.kblocks, 0, false};
  uint64_t d_base = 0;
  if (p.mode == kGroupedRows) {
    part = find_rows<BM>(p, tm);
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
  const uint64_t pitch = static_cast<uint64_t>(p.kblocks) * kBlock;
  const uint8_t *a = p.a + m0 * pitch, *b = p.b + n0 * pitch;
  const float *sa = p.sa + m0, *sb = p.sb;
  if (p.mode == kGroupedRows) {
    b += static_cast<uint64_t>(part.group) * p.n * pitch;
    sb += static_cast<uint64_t>(part.group) * p.sb_stride * p.kblocks;
  }

  // where this lane's share of each load comes from: rows past the end repeat the last one
  const uint32_t chunk = lane % 8;
  const uint32_t phase = PHASED ? wave / (kWaves / 2) : 0, quarter = wave % (kWaves / 2);
  uint32_t from_a[kLoadA], from_b[PHASED ? 2 : kLoadB];
#pragma unroll
  for (uint32_t i = 0; i < kLoadA; ++i) {
    const uint32_t r = (wave * kLoadA + i) * 8 + lane / 8;
    from_a[i] = min(r, part.m_end - 1 - m0) * static_cast<uint32_t>(pitch) + ((chunk ^ (r & 7)) << 4);
  }
#pragma unroll
  for (uint32_t i = 0; i < (PHASED ? 2 : kLoadB); ++i) {
    // (phased: n is a multiple of BN, and rows go up by whole pitches; by G the swizzle may take turns every eight rows)
    const uint32_t r = PHASED ? (quarter * 2 * kLoadB + i) * 8 + lane / 8 : (wave * kLoadB + i) * 8 + lane / 8;
    from_b[i] = min(r, p.n - 1 - n0) * static_cast<uint32_t>(pitch) + ((chunk ^ swizzle_b<G>(r)) << 4);
  }
  if (SBV) sb += n0;
  // scales: 64 at a time, of 64 rows of a or of b; of b in 128x128 blocks, 64 times its block's.
  // (Where there are more waves than that, some load the same again.)
  uint32_t from_s[PHASED ? 2 : kLoadS];
#pragma unroll
  for (uint32_t i = 0; i < (PHASED ? 2 : kLoadS); ++i) {
    const uint32_t w = PHASED ? (i == 0 ? phase * (BM / 128) + quarter % (BM / 128) : BM / 64 + quarter) : (wave * kLoadS + i) % kGroups, r = (w < BM / 64 ? w : w - BM / 64) * 64 + lane;
    from_s[i] = 4 * (w < BM / 64 ? min(r, part.m_end - 1 - m0) : SBV ? min(r, p.n - 1 - n0) : min((n0 + r) / kBlock, p.sb_stride - 1));
  }

  const uint32_t lds_data = lds_address(&lds[share][0][0]), lds_scales = lds_address(&scales[share][0][0]);
  auto load = [&](uint32_t kb, uint32_t stage) {
    const uint8_t *ka = a + static_cast<uint64_t>(kb) * kBlock, *kbp = b + static_cast<uint64_t>(kb) * kBlock;
    const uint32_t to = lds_data + stage * static_cast<uint32_t>(sizeof lds[0][0]);
#pragma unroll
    for (uint32_t i = 0; i < kLoadA; ++i) load16_to_lds(to + (wave * kLoadA + i) * 1024, ka, from_a[i]);
#pragma unroll
    for (uint32_t i = 0; i < (PHASED ? 0 : kLoadB); ++i) load16_to_lds(to + BM * kBlock + (wave * kLoadB + i) * 1024, kbp, from_b[i]);
    if (PHASED && phase == 0) {
#pragma unroll
      for (uint32_t i = 0; i < 2 * kLoadB; ++i)
        load16_to_lds(to + BM * kBlock + (quarter * 2 * kLoadB + i) * 1024, kbp + (G == 1 ? i : i / 2 * 2) * 8 * pitch, from_b[G == 1 ? 0 : i % 2]);
    }
#pragma unroll
    for (uint32_t i = 0; i < (PHASED ? 2 : kLoadS); ++i) {
      const uint32_t w = PHASED ? (i == 0 ? phase * (BM / 128) + quarter % (BM / 128) : BM / 64 + quarter) : (wave * kLoadS + i) % kGroups;
      if (PHASED && (i == 0 ? quarter >= BM / 128 : phase == 1)) continue;
      load4_to_lds(lds_scales + stage * static_cast<uint32_t>(sizeof scales[0][0]) + w * 256,
                   w < BM / 64 ? sa + static_cast<uint64_t>(kb) * p.sa_stride : sb + static_cast<uint64_t>(kb) * p.sb_stride, from_s[i]);
    }
  };

  const uint32_t wm = PHASED ? phase : wave % WM, wn = PHASED ? quarter : wave / WM;
  const bool active = m0 + wm * TM < part.m_end;  // a phased tile's lower half may have no rows: its waves then only load and wait
  const uint32_t i16 = lane % 16, q = lane / 16;
  f32x4 acc[MI][NI];
#pragma unroll
  for (uint32_t i = 0; i < MI; ++i)
#pragma unroll
    for (uint32_t j = 0; j < NI; ++j) acc[i][j] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};

  // a row's chunks q and q + 4 are this lane's 32 bytes of it: a and b share
  // that order along k, and inside a block the order of the sum is free
  auto chunk_at = [&](const uint8_t *base, uint32_t r, uint32_t g, uint32_t f) {
    return *reinterpret_cast<const u32x4 *>(base + r * kBlock + ((g ^ f) << 4));
  };

  // The lanes that met scales that are not near(): with any, the wave's sums do not count.
  uint64_t far = 0;
  const uint32_t look = PHASED ? 0 : lane % TM;
  auto look_at_scales = [&](const float *ls, float sbu) {
    uint32_t l = look;
    if (PHASED) {  // the lane's number anew, so that it holds no register through the steps
      uint32_t all = ~0u;
      asm volatile("" : "+s"(all));
      l = __builtin_amdgcn_mbcnt_hi(all, __builtin_amdgcn_mbcnt_lo(all, 0));
    }
    bool ok = true;
#pragma unroll
    for (uint32_t i = 0; i < TM; i += kWave) ok = ok & near<SBV>(ls[i + l], sbu);
    far |= __ballot(!ok);
  };

  auto step = [&](uint32_t stage) {
    const uint8_t *la = &lds[share][stage][wm * TM * kBlock], *lb = &lds[share][stage][(BM + wn * TN) * kBlock];
    const float *ls = &scales[share][stage][wm * TM], *lsb = &scales[share][stage][BM + wn * TN];
    const float sbu = SBV ? 1.0f : lsb[0];  // its columns are in one 128x128 block of b
    look_at_scales(ls, sbu);
    Wide b0[NI], b1[NI];
    f32x4 sbv[NI];
#pragma unroll
    for (uint32_t j = 0; j < NI; ++j) {
      const uint32_t r = (j / G) * 16 * G + (i16 / 4) * 4 * G + (j % G) * 4 + i16 % 4;
      const uint32_t f = i16 & 7;  // f(r): r's low two bits and the lowest bit of i16 / 4
      b0[j] = widen(chunk_at(lb, r, q, f));
      b1[j] = widen(chunk_at(lb, r, q + 4, f));
      if (SBV) sbv[j] = *reinterpret_cast<const f32x4 *>(lsb + (j / G) * 16 * G + q * 4 * G + (j % G) * 4);
    }
#pragma unroll
    for (uint32_t i = 0; i < MI; ++i) {
      if (PHASED && i == kTurn) lds_barrier();
      const Wide a0 = widen(chunk_at(la, i * 16 + i16, q, i16 & 7)), a1 = widen(chunk_at(la, i * 16 + i16, q + 4, i16 & 7));
      const float s = ls[i * 16 + i16];
#pragma unroll
      for (uint32_t j = 0; j < NI; ++j) {
        const f32x4 c = block_sum(b0[j], b1[j], a0, a1);
#pragma unroll
        for (uint32_t e = 0; e < 4; ++e) acc[i][j][e] = SBV ? __builtin_fmaf(c[e] * s, sbv[j][e], acc[i][j][e]) : __builtin_fmaf(c[e], s * sbu, acc[i][j][e]);
      }
    }
  };

  // The same with its instructions in an order of its own (the scheduler's has
  // the matrix cores wait for the next fragment, and for sums of four dependent
  // products; 8192 x 8192 x 5120 in 256x256 tiles took 535 us so, and takes
  // 500): groups of two v_mfma of different tiles, each group with at most eight
  // vector instructions beside it. Those widen half of the next fragment, or
  // scale tiles whose products ended a group before.
  auto step_in_groups = [&](uint32_t stage) {
    if constexpr (kGrouped) {
      const uint8_t *la = &lds[share][stage][wm * TM * kBlock], *lb = &lds[share][stage][(BM + wn * TN) * kBlock];
      const float *ls = &scales[share][stage][wm * TM], *lsb = &scales[share][stage][BM + wn * TN];
      const float sbu = SBV ? 1.0f : lsb[0];
      look_at_scales(ls, sbu);
      f32x4 sbv[NI];
      const uint32_t f = i16 & 7;
      u32x4 lo = chunk_at(la, i16, q, f), hi = chunk_at(la, i16, q + 4, f);  // a's fragment, as loaded
      float s = SBV ? ls[i16] : ls[i16] * sbu, s_next = 0.0f;
      Wide b0[NI], b1[NI], a0 = widen(lo), a1;
#pragma unroll
      for (uint32_t j = 0; j < NI; ++j) {
        const uint32_t r = (j / G) * 16 * G + (i16 / 4) * 4 * G + (j % G) * 4 + i16 % 4;
        b0[j] = widen(chunk_at(lb, r, q, f));
        b1[j] = widen(chunk_at(lb, r, q + 4, f));
        if (SBV) sbv[j] = *reinterpret_cast<const f32x4 *>(lsb + (j / G) * 16 * G + q * 4 * G + (j % G) * 4);
      }
      f32x4 c[4];
      auto product = [&](uint32_t j, const bf16x8 &x, const bf16x8 &y, bool first) {
        c[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(x, y, first ? f32x4{0.0f, 0.0f, 0.0f, 0.0f} : c[j], 0, 0, 0);
      };
      auto scale = [&](uint32_t i, uint32_t j, float by) {
#pragma unroll
        for (uint32_t e = 0; e < 4; ++e) acc[i][j][e] = SBV ? __builtin_fmaf(c[j][e] * by, sbv[j][e], acc[i][j][e]) : __builtin_fmaf(c[j][e], by, acc[i][j][e]);
      };
      float s_last = 0.0f;
#pragma unroll
      for (uint32_t i = 0; i < MI; ++i) {
        if (PHASED && i == kTurn) lds_barrier();
        const bool more = i + 1 < MI;
        product(0, b0[0].lo, a0.lo, true);
        product(1, b0[1].lo, a0.lo, true);
        a1.lo = widen8(hi.x, hi.y);
        __builtin_amdgcn_sched_barrier(0);
        product(0, b0[0].hi, a0.hi, false);
        product(1, b0[1].hi, a0.hi, false);
        a1.hi = widen8(hi.z, hi.w);
        if (more) {
          lo = chunk_at(la, (i + 1) * 16 + i16, q, f);
          hi = chunk_at(la, (i + 1) * 16 + i16, q + 4, f);
          s_next = ls[(i + 1) * 16 + i16];
        }
        __builtin_amdgcn_sched_barrier(0);
        product(0, b1[0].lo, a1.lo, false);
        product(1, b1[1].lo, a1.lo, false);
        if (i > 0) scale(i - 1, 2, s_last);
        __builtin_amdgcn_sched_barrier(0);
        product(0, b1[0].hi, a1.hi, false);
        product(1, b1[1].hi, a1.hi, false);
        if (i > 0) scale(i - 1, 3, s_last);
        __builtin_amdgcn_sched_barrier(0);
        product(2, b0[2].lo, a0.lo, true);
        product(3, b0[3].lo, a0.lo, true);
        __builtin_amdgcn_sched_barrier(0);
        product(2, b0[2].hi, a0.hi, false);
        product(3, b0[3].hi, a0.hi, false);
        scale(i, 0, s);
        __builtin_amdgcn_sched_barrier(0);
        product(2, b1[2].lo, a1.lo, false);
        product(3, b1[3].lo, a1.lo, false);
        scale(i, 1, s);
        if (more) a0.lo = widen8(lo.x, lo.y);
        __builtin_amdgcn_sched_barrier(0);
        product(2, b1[2].hi, a1.hi, false);
        product(3, b1[3].hi, a1.hi, false);
        if (more) a0.hi = widen8(lo.z, lo.w);
        s_last = s;
        s = SBV ? s_next : s_next * sbu;
        __builtin_amdgcn_sched_barrier(0);
      }
      scale(MI - 1, 2, s_last);
      scale(MI - 1, 3, s_last);
    }
  };

  if (KS > 1 && threadIdx.x < kWaves) far_waves[threadIdx.x] = false;  // read and written past a barrier
  if (!part.zero && part.kb0 < part.kb_end) {
    // (a share without a block in the last round loads the last one and leaves it)
    const uint32_t last = part.kb_end - 1;
    load(min(part.kb0 + share, last), 0);
    if (PHASED && phase == 1) lds_barrier();
    uint32_t stage = 0;
    for (uint32_t first = part.kb0; first < part.kb_end; first += KS) {
      wait_loads();   // this step's loads are in,
      lds_barrier();  // everyone's are, and everyone has read the other stage
      if (first + KS < part.kb_end) load(min(first + KS + share, last), stage ^ 1);
      if (KS == 1 || first + share < part.kb_end) {
        if (PHASED && !active) lds_barrier();
        else if (kGrouped) step_in_groups(stage);
        else step(stage);
      }
      stage ^= 1;
    }
    if (PHASED && phase == 0) lds_barrier();
  }

  // The wave's part of the tile from memory, 16x16 sums at a time, all blocks along k: add_far()'s way.
  auto far_tile = [&] {
#pragma unroll 1
    for (uint32_t i = 0; i < MI; ++i) {
      const uint32_t row = wm * TM + i * 16 + i16, ra = min(row, part.m_end - 1 - m0);
#pragma unroll 1
      for (uint32_t j = 0; j < NI; ++j) {
        const uint32_t col = wn * TN + j * 16, rb = min(col + i16, p.n - 1 - n0);
        f32x4 v{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 2
        for (uint32_t kb = part.kb0; kb < part.kb_end; ++kb) {
          const uint64_t at = static_cast<uint64_t>(kb) * kBlock + 16 * q;
          const u32x4 *pa = reinterpret_cast<const u32x4 *>(a + ra * pitch + at), *pb = reinterpret_cast<const u32x4 *>(b + rb * pitch + at);
          const float *ps = sb + static_cast<uint64_t>(kb) * p.sb_stride;
          f32x4 s;
#pragma unroll
          for (uint32_t e = 0; e < 4; ++e) s[e] = ps[SBV ? min(col + 4 * q + e, p.n - 1 - n0) : min((n0 + col) / kBlock, p.sb_stride - 1)];
          v = add_far(v, block_sum(widen(pb[0]), widen(pb[4]), widen(pa[0]), widen(pa[4])), sa[static_cast<uint64_t>(kb) * p.sa_stride + ra], s);
        }
        const uint32_t m = m0 + row;
        if (m < part.m_end) store4<OUT32>(p.d, d_base + static_cast<uint64_t>(m) * p.n, n0 + col + 4 * q, p.n, v);
      }
    }
  };

  if (KS > 1) {  // the shares' sums meet in the first one's registers, in their order
    f32x4(*sums)[MI * NI][kWaves][kWave] = reinterpret_cast<f32x4(*)[MI * NI][kWaves][kWave]>(&lds[0][0][0]);
    static_assert((KS - 1) * sizeof sums[0] <= sizeof lds, "the sums fit the stages");
    lds_barrier();
    if (share > 0) {
      if (far != 0) far_waves[wave] = true;
#pragma unroll
      for (uint32_t i = 0; i < MI; ++i)
#pragma unroll
        for (uint32_t j = 0; j < NI; ++j) sums[share - 1][i * NI + j][wave][lane] = acc[i][j];
    }
    lds_barrier();
    if (share > 0) return;
    if (far_waves[wave]) far = 1;
#pragma unroll
    for (uint32_t k = 0; k + 1 < KS; ++k)
#pragma unroll
      for (uint32_t i = 0; i < MI; ++i)
#pragma unroll
        for (uint32_t j = 0; j < NI; ++j) acc[i][j] += sums[k][i * NI + j][wave][lane];
  }

  if (far != 0) {
    far_tile();
    return;
  }
#pragma unroll
  for (uint32_t i = 0; i < MI; ++i) {
    const uint32_t m = m0 + wm * TM + i * 16 + i16;
    if (m >= part.m_end) continue;
    const uint64_t row = d_base + static_cast<uint64_t>(m) * p.n;
#pragma unroll
    for (uint32_t g = 0; g < NG; ++g) {
      float v[4 * G];
#pragma unroll
      for (uint32_t e = 0; e < 4 * G; ++e) v[e] = acc[i][G * g + e / 4][e % 4];
      store<OUT32, 4 * G>(p.d, row, n0 + wn * TN + 16 * G * g + 4 * G * q, p.n, v);
    }
  }
}

// ---------------------------------------------------------------------------
// Few rows: tiles of up to kRowsM rows and kRowsN columns, the blocks along k
// dealt out to the KS waves of a workgroup, each with accumulators of its own,
// which meet in LDS at the end, in the order of the waves. Operands go from
// memory to registers, U blocks of them asked for before the first is used:
// each row of b is read once and by one wave, so LDS would only add a step.
// ---------------------------------------------------------------------------
constexpr uint32_t kRowsM = 64, kRowsN = 32;

template <uint32_t KS, uint32_t MT, uint32_t U, bool SBV, bool OUT32>
__device__ __forceinline__ void rows_tile(const Args &p, const Part &part, const uint8_t *a, const uint8_t *b, const float *sa,
                                          const float *sb, uint32_t n0, f32x4 (*red)[kRowsM / 16 * 2][kWave]) {
  const uint32_t lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const uint32_t i16 = lane % 16, q = lane / 16;
  const uint32_t pitch = p.kblocks * kBlock;
  // tile t of b takes rows 8 (i / 4) + 4 t + i % 4, so that a lane ends with 8 consecutive columns of d
  uint32_t at_a[MT], at_b[2], row_a[MT];
#pragma unroll
  for (uint32_t i = 0; i < MT; ++i) {
    row_a[i] = min(16 * i + i16, part.m_end - 1 - part.m0);
    at_a[i] = row_a[i] * pitch + 16 * q;
  }
#pragma unroll
  for (uint32_t t = 0; t < 2; ++t) at_b[t] = min(8 * (i16 / 4) + 4 * t + i16 % 4, p.n - 1 - n0) * pitch + 16 * q;
  uint32_t row_sb[2][4];
  if (SBV) {
#pragma unroll
    for (uint32_t t = 0; t < 2; ++t)
#pragma unroll
      for (uint32_t e = 0; e < 4; ++e) row_sb[t][e] = min(8 * q + 4 * t + e, p.n - 1 - n0);
  }
  const uint32_t nb = n0 / kBlock;

  f32x4 acc[MT][2];
#pragma unroll
  for (uint32_t i = 0; i < MT; ++i) acc[i][0] = acc[i][1] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  for (uint32_t kb0 = part.kb0 + wave; kb0 < part.kb_end; kb0 += U * KS) {
    u32x4 wa[U][MT][2], wb[U][2][2];
    float fa[U][MT], fb[U][2][4];
#pragma unroll
    for (uint32_t u = 0; u < U; ++u) {
      const uint32_t kb = min(kb0 + u * KS, part.kb_end - 1);  // past the end: loaded again, not used
      const uint8_t *ka = a + static_cast<uint64_t>(kb) * kBlock, *kbp = b + static_cast<uint64_t>(kb) * kBlock;
#pragma unroll
      for (uint32_t t = 0; t < 2; ++t) {
        wb[u][t][0] = *reinterpret_cast<const u32x4 *>(kbp + at_b[t]);
        wb[u][t][1] = *reinterpret_cast<const u32x4 *>(kbp + at_b[t] + 64);
      }
#pragma unroll
      for (uint32_t i = 0; i < MT; ++i) {
        wa[u][i][0] = *reinterpret_cast<const u32x4 *>(ka + at_a[i]);
        wa[u][i][1] = *reinterpret_cast<const u32x4 *>(ka + at_a[i] + 64);
        fa[u][i] = sa[static_cast<uint64_t>(kb) * p.sa_stride + row_a[i]];
      }
      if (SBV) {
#pragma unroll
        for (uint32_t t = 0; t < 2; ++t)
#pragma unroll
          for (uint32_t e = 0; e < 4; ++e) fb[u][t][e] = sb[static_cast<uint64_t>(kb) * p.sb_stride + n0 + row_sb[t][e]];
      } else {
        fb[u][0][0] = sb[static_cast<uint64_t>(kb) * p.sb_stride + nb];
      }
    }
#pragma unroll
    for (uint32_t u = 0; u < U; ++u) {
      if (kb0 + u * KS >= part.kb_end) break;
      Wide b0[2], b1[2];
#pragma unroll
      for (uint32_t t = 0; t < 2; ++t) {
        b0[t] = widen(wb[u][t][0]);
        b1[t] = widen(wb[u][t][1]);
      }
#pragma unroll
      for (uint32_t i = 0; i < MT; ++i) {
        const Wide a0 = widen(wa[u][i][0]), a1 = widen(wa[u][i][1]);
#pragma unroll
        for (uint32_t t = 0; t < 2; ++t) {
          const float *f = fb[u][SBV ? t : 0];
          acc[i][t] = add_far(acc[i][t], block_sum(b0[t], b1[t], a0, a1), fa[u][i],
                              SBV ? f32x4{f[0], f[1], f[2], f[3]} : f32x4{f[0], f[0], f[0], f[0]});
        }
      }
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

template <uint32_t KS, bool SBV, bool OUT32>
__global__ __launch_bounds__(KS *kWave) void k_fp8_rows(Args p) {
  __shared__ f32x4 red[KS][kRowsM / 16 * 2][kWave];
  const uint32_t tn = blockIdx.x % p.tiles_n, tm = blockIdx.x / p.tiles_n;
  Part part{tm * kRowsM, min(p.m, (tm + 1) * kRowsM), 0, p.kblocks, 0, false};
  if (p.mode == kGroupedRows) {
    part = find_rows<kRowsM>(p, tm);
    if (part.m0 >= part.m_end) return;
    part.m_end = min(part.m_end, part.m0 + kRowsM);
    if (part.zero) part.kb_end = 0;
  }
  const uint32_t n0 = tn * kRowsN;
  const uint64_t pitch = static_cast<uint64_t>(p.kblocks) * kBlock;
  const uint8_t *a = p.a + part.m0 * pitch, *b = p.b + n0 * pitch;
  const float *sa = p.sa + part.m0, *sb = p.sb;
  if (p.mode == kGroupedRows) {
    b += static_cast<uint64_t>(part.group) * p.n * pitch;
    sb += static_cast<uint64_t>(part.group) * p.sb_stride * p.kblocks;
  }
  const uint32_t rows = part.m_end - part.m0;
  if (rows <= 16) rows_tile<KS, 1, 4, SBV, OUT32>(p, part, a, b, sa, sb, n0, red);
  else if (rows <= 32) rows_tile<KS, 2, 2, SBV, OUT32>(p, part, a, b, sa, sb, n0, red);
  else rows_tile<KS, 4, 2, SBV, OUT32>(p, part, a, b, sa, sb, n0, red);  // a group's, above the average
}

template <uint32_t KS>
hipError_t launch_rows(const Fp8Matmul &p, hipStream_t s) {
  Args a{p.a, p.b, p.sa, p.sb, p.d, p.m, p.n, p.kblocks, p.sa_stride, p.sb_stride, p.mode, p.offsets, p.groups, 0, 0};
  a.tiles_n = (p.n + kRowsN - 1) / kRowsN;
  a.tiles_m = p.mode == kGroupedRows ? p.m / kRowsM + p.groups + 1 : (p.m + kRowsM - 1) / kRowsM;
  const uint64_t blocks = static_cast<uint64_t>(a.tiles_m) * a.tiles_n;
  if (blocks * KS * kWave >= kMaxThreads1D) return hipErrorInvalidConfiguration;
  const dim3 grid(static_cast<uint32_t>(blocks)), threads(KS * kWave);
  if (p.b_block_2d) {
    if (p.out_fp32) hipLaunchKernelGGL((k_fp8_rows<KS, false, true>), grid, threads, 0, s, a);
    else hipLaunchKernelGGL((k_fp8_rows<KS, false, false>), grid, threads, 0, s, a);
  } else {
    if (p.out_fp32) hipLaunchKernelGGL((k_fp8_rows<KS, true, true>), grid, threads, 0, s, a);
    else hipLaunchKernelGGL((k_fp8_rows<KS, true, false>), grid, threads, 0, s, a);
  }
  return hipGetLastError();
}

template <uint32_t BM, uint32_t BN, uint32_t WM, uint32_t WN, uint32_t KS = 1, bool PHASED = false>
hipError_t launch_tile(const Fp8Matmul &p, hipStream_t s) {
  Args a{p.a, p.b, p.sa, p.sb, p.d, p.m, p.n, p.kblocks, p.sa_stride, p.sb_stride, p.mode, p.offsets, p.groups, 0, 0};
  a.tiles_n = (p.n + BN - 1) / BN;
  a.tiles_m = (p.m + BM - 1) / BM;
  uint64_t rows = a.tiles_m;
  // every group may end in a partial tile, and so may the rows past the last one
  if (p.mode == kGroupedRows) rows = p.m / BM + p.groups + 1;
  if (p.mode == kGroupedK) rows = static_cast<uint64_t>(a.tiles_m) * p.groups;
  const uint64_t blocks = rows * a.tiles_n;
  if (blocks * WM * WN * KS * kWave >= kMaxThreads1D) return hipErrorInvalidConfiguration;
  const dim3 grid(static_cast<uint32_t>(blocks)), threads(WM * WN * KS * kWave);
  if (p.b_block_2d) {
    if (p.out_fp32) hipLaunchKernelGGL((k_fp8_tile<BM, BN, WM, WN, KS, PHASED, false, true>), grid, threads, 0, s, a);
    else hipLaunchKernelGGL((k_fp8_tile<BM, BN, WM, WN, KS, PHASED, false, false>), grid, threads, 0, s, a);
  } else {
    if (p.out_fp32) hipLaunchKernelGGL((k_fp8_tile<BM, BN, WM, WN, KS, PHASED, true, true>), grid, threads, 0, s, a);
    else hipLaunchKernelGGL((k_fp8_tile<BM, BN, WM, WN, KS, PHASED, true, false>), grid, threads, 0, s, a);
  }
  return hipGetLastError();
}

}  // namespace

// Which kernel. Times in us, of one session.
//   Few rows, against the 64x64 tiles below: m up to 32:
//     16 x 8192 x 5120        9.9 / 16.7         32 x 4096 x 4096  10.3 / 13.6
//     32 x 8192 x 5120       12.5 / 17.0;  but   64 x 8192 x 5120  17.7 / 17.2
//   or up to 32 a group on average, by the buffer's rows, against 128x128 tiles:
//     64 groups, 1472 rows x 4096 x 2048  106 / 130     52 groups, 1280 rows  90 / 112
//     32 groups,  992 rows x 4096 x 2048   56 / 63      the same x 2048 x 2048  31 / 33
//     64 groups, 1792 rows x 4096 x 2048  147 / 154;  at 2048 rows both 157
//   Up to 160 tiles of 128x128 they leave CUs idle, and a wave that has its
//   SIMD to itself takes 0.5 us a step, most of it waiting for its own last
//   instruction. So up to 256 tiles of 64x64 (one a CU) those, with 16 waves in
//   four shares of the blocks along k, against four waves and against 128x128:
//     256 x 4096 x 4096       15.3 / 20.0 / 40   256 x 1024 x 8192  24 / 36 / 75
//   and above that 64x128 tiles with 8 waves in two shares, against 64x64 with four waves:
//     777 x 1361 x 1999       15.1 / 16.1        512 x 4096 x 4096  24 / 27
//     but 1280 x 2048 x 4096 (160 tiles of 128x128)  43 / 35, and 128x128 40;
//     1024 x 4096 x 2048 (256 tiles of 128x128)  24.6, and 128x128, which it takes, 23.4
//   256x256 tiles, phased, where their rounds over 256 CUs, 3.1 us a step along
//   k, take less than those of 128x128 tiles over 512 places, 1.8 us a step:
//     8192 x 8192 x 5120      516 / 607          4096 x 4096 x 4096  107 / 126
//     8 groups, 66432 rows x 4096 x 2048  905 / 1015    16 groups, 34688 rows x 2048 x 4096  495 / 546
//     64 groups, 73600 rows x 4096 x 2048  1029 / 1126  32 weight gradients of 4096 x 2048  699 / 713
//     but 16 weight gradients of 2048 x 2048  202 / 185: a tile's stores weigh more with nine steps;
//     3000 x 8192 x 5120, which takes 128x128, 238 / 240, and 2560 rows 236 / 206
hipError_t launch_fp8_matmul(const Fp8Matmul &p, hipStream_t s) {
  const bool few = p.mode == kDense ? p.m <= 32 : p.mode == kGroupedRows && p.m <= 32 * static_cast<uint64_t>(p.groups);
  if (few) {
    // a wave's share is best at least the four blocks that it asks for at once
    if (p.kblocks >= 24) return launch_rows<8>(p, s);
    if (p.kblocks >= 12) return launch_rows<4>(p, s);
    if (p.kblocks >= 6) return launch_rows<2>(p, s);
    return launch_rows<1>(p, s);
  }
  // by groups of rows, every second group's last tile is taken to be a partial one
  auto count = [&](uint64_t edge) {
    const uint64_t rows = (p.m + edge - 1) / edge + (p.mode == kGroupedRows ? p.groups / 2 : 0);
    return rows * ((p.n + edge - 1) / edge) * (p.mode == kGroupedK ? p.groups : 1);
  };
  const uint64_t tiles = count(128);
  if (tiles <= 160) return count(64) <= 256 ? launch_tile<64, 64, 2, 2, 4>(p, s) : launch_tile<64, 128, 2, 2, 2>(p, s);
  if (p.n % 256 == 0 && 64 * ((count(256) + 255) / 256) <= 37 * ((tiles + 511) / 512))
    return launch_tile<256, 256, 2, 4, 1, true>(p, s);
  return launch_tile<128, 128, 2, 2>(p, s);
}

}  // namespace nvfp4
