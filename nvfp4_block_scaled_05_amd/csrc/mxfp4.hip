// MXFP4: E2M1 codes with one E8M0 scale (a power of two) for each 32 values
// along a row (or each 32x32), in the row-wise and the column-wise (transposed)
// orientation from one read of the input, and the way back.
//
//   m = max|v| of the block, E its exponent field in binary32
//   s = max(E - 2, 0); 255 (NaN) where E is 255, an infinity or a NaN
//   X = 2^(s - 127); code = E2M1(v / X), nearest even, at most 6; 0 where s is 255
//
// which is 2^(floor(log2 m) - 2), clamped at 2^-127: |v / X| < 8, and what is
// above 6 becomes 6. The gfx950 conversions to E2M1 divide by X and round
// once; BF16 goes in as it is, two values a word, with no multiplication or
// widening of its own (36736 gathered rows both ways 111 -> 97 us, the input in the Infinity Cache).
//
// One workgroup per 128x128 tile, in registers: thread t holds the 8x8 patch
// at rows 8 (t / 16), columns 8 (t % 16). Four neighbouring lanes hold a row's
// block of 32 and a wave holds 32 rows, so every maximum stays inside a wave.
// A patch's 8 codes of a row (of a column) are one word; the words pass
// through LDS so that they leave 16 bytes a lane, 64 contiguous bytes a row.
// Columns and rows past the end count as zeros; each orientation's rows are
// padded to a multiple of 128 with zero codes, which every tile writes whole.
// Bound by HBM: 2 (or 4) bytes read and half a byte a side written for each value.
// 32 x 2048x4096 BF16 in 2D both ways takes 163 us, 5.0 TB/s, where a copy of 1 GiB on
// the same card moves 5.1, FP32 285 us, 4.8; reading it back to BF16 132 us, 5.2 TB/s, to FP32 261, 4.7.
#include "codec.h"
#include "launch.h"
#include "patch.h"

namespace nvfp4 {
namespace {

constexpr uint32_t kThreads = 256;
constexpr uint32_t kTile = kFp8Block;
constexpr uint32_t kPerWord = kTile / 8;  // words of a tile's row of codes

// Inputs that the Infinity Cache (256 MB) is likely to hold, and gathered rows, which are read several times, are kept
// there: the outputs are stored past the caches. 8192x5120 BF16 both ways 29.8 -> 26.6 us, 36736 gathered rows of
// 5120 columns both ways 118 -> 97 (call after call on one input; 116 to 123 where other calls come between); but
// 8192x8192 47 -> 53 and 32 x 2048x4096 163 -> 169, which are not.
constexpr uint64_t kStreamBelow = uint64_t{1} << 27;
// For the others a workgroup asks for LDS that it does not use, so that six are on a CU, not eight, whose reads and stores
// are too far apart: 32 x 2048x4096 both ways 180 us with eight, 171 with seven, 163 with six, 173 with five, 172 with four.
constexpr uint32_t kIdleLds = 7680;

struct Args {
  const void *x;
  uint32_t rows, cols;             // of one matrix
  uint32_t row_tiles, col_tiles;
  uint32_t tiles;                  // of all matrices
  const int32_t *row_slots;
  uint32_t slots, topk;
  uint8_t *row_data, *col_data;
  uint32_t *row_scales, *col_scales;  // four blocks a word
};

// The scale byte of a block from its largest magnitude's bits.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax_bits) {
  const uint32_t e = amax_bits >> 23;
  return e == 255 ? 255 : e > 2 ? e - 2 : 0;
}
// The codes of eight values, in a row's or a column's order, of a block with scale byte s. The conversions divide by a
// power of two, whose exponent field they take from the scale as the byte is (0: 2^-127), exactly, and round once.
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t encode(const uint32_t *pairs, uint32_t s) {
  const float x = __uint_as_float(s << 23);
  uint32_t w = pairs[0];  // (all of it is written)
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2, pairs[0]), x, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2, pairs[1]), x, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2, pairs[2]), x, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(bf16x2, pairs[3]), x, 3);
  return s == 255 ? 0 : w;
}
__device__ __forceinline__ uint32_t encode(const float *v, uint32_t s) {
  const float x = __uint_as_float(s << 23);
  uint32_t w = __float_as_uint(v[0]);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], x, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], x, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], x, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], x, 3);
  return s == 255 ? 0 : w;
}
__device__ __forceinline__ uint32_t encode_row(const Patch<kBF16> &v, int p, uint32_t s) {
  const uint32_t pairs[4] = {v.w[p][0], v.w[p][1], v.w[p][2], v.w[p][3]};
  return encode(pairs, s);
}
__device__ __forceinline__ uint32_t encode_col(const Patch<kBF16> &v, int q, uint32_t s) {
  uint32_t pairs[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) pairs[i] = __builtin_amdgcn_perm(v.w[2 * i + 1][q / 2], v.w[2 * i][q / 2], q % 2 ? 0x07060302 : 0x05040100);
  return encode(pairs, s);
}
__device__ __forceinline__ uint32_t encode_row(const Patch<kFP32> &v, int p, uint32_t s) { return encode(v.v[p], s); }
__device__ __forceinline__ uint32_t encode_col(const Patch<kFP32> &v, int q, uint32_t s) {
  float f[8];
#pragma unroll
  for (int p = 0; p < 8; ++p) f[p] = v.v[p][q];
  return encode(f, s);
}

// Where the word of row i and column group g of a tile is: eight rows take 16
// words more than they fill, and groups of four words are swapped by pairs of eights,
// so that a wave's 16 column groups of four rows, and its four row groups of
// 16 columns of the transposed tile, meet every bank twice, which 64 lanes must.
constexpr uint32_t kEight = 9 * kPerWord;
__device__ __forceinline__ uint32_t place(uint32_t i, uint32_t g) { return i / 8 * kEight + i % 8 * kPerWord + (g ^ (i / 16 % 4 * 4)); }

template <int DT, bool BLOCK_2D, bool STREAM>
__global__ __launch_bounds__(kThreads) void k_mxfp4_quantize(Args a) {
  __shared__ __attribute__((aligned(16))) uint32_t straight[kTile / 8 * kEight], turned[kTile / 8 * kEight];
  __shared__ __attribute__((aligned(4))) uint8_t col_bytes[kTile][4];
  const uint32_t t = threadIdx.x, cg = t % 16, rg = t / 16, lane = t % 64, wave = t / 64;
  const uint32_t block = block_of_long_grid();
  if (block >= a.tiles) return;
  const uint32_t per_batch = a.row_tiles * a.col_tiles, batch = block / per_batch, id = block - batch * per_batch;
  // Workgroups go to the eight XCDs in turn. Two tiles that share the cache lines of a row's codes go to one, after each
  // other, and so do all that share the lines of a column's; a gathered row, read topk times, stays in its L2 too.
  const uint32_t strip = id / (16 * a.row_tiles) * 16, in = id - strip * a.row_tiles, wide = min(16u, a.col_tiles - strip);
  uint32_t ct = strip + in % wide, rt = in / wide;
  if (wide == 16) ct = strip + in % 8 * 2 + in / 8 % 2;
  const uint32_t r0 = rt * kTile, c0 = ct * kTile;
  const uint32_t c = c0 + 8 * cg;
  const uint32_t left = c < a.cols ? a.cols - c : 0;

  Patch<DT> v;
#pragma unroll
  for (uint32_t p = 0; p < 8; ++p) {
    const uint32_t r = r0 + 8 * rg + p;
    bool have = r < a.rows && left > 0;
    uint64_t src = static_cast<uint64_t>(batch) * a.rows + r;
    if (a.row_slots != nullptr && have) {
      const uint32_t slot = static_cast<uint32_t>(a.row_slots[r]);
      have = slot < a.slots;
      src = slot / a.topk;
    }
    if (have) v.load(p, a.x, src * a.cols + c, left);
    else v.clear(p);
  }

  const bool want_row = a.row_data != nullptr, want_col = a.col_data != nullptr;
  uint32_t col_max[8];
  if (BLOCK_2D || want_col) v.col_max(col_max);  // over the wave's 32 rows
  uint32_t both = 0;
  if (BLOCK_2D) {
    uint32_t m = col_max[0];
#pragma unroll
    for (int q = 1; q < 8; ++q) m = max(m, col_max[q]);
    m = max(m, dpp_mov<kQuadXor1>(m));
    both = scale_byte(max(m, dpp_mov<kQuadXor2>(m)));
  }

  if (want_row) {
    uint32_t mine = 0;  // the scale word of row cg of the patch
#pragma unroll
    for (uint32_t p = 0; p < 8; ++p) {
      uint32_t s = both;
      if (!BLOCK_2D) {
        uint32_t m = v.row_max(p);
        m = max(m, dpp_mov<kQuadXor1>(m));
        s = scale_byte(max(m, dpp_mov<kQuadXor2>(m)));
      }
      uint32_t w = s << (8 * (cg / 4));  // the row's four blocks: the other quads', by mirrors
      w |= dpp_mov<0x141>(w);
      w |= dpp_mov<0x140>(w);
      mine = cg == p ? w : mine;
      straight[place(8 * rg + p, cg)] = encode_row(v, p, s);
    }
    const uint32_t r = r0 + 8 * rg + cg;
    if (cg < 8 && r < a.rows) a.row_scales[(static_cast<uint64_t>(batch) * a.col_tiles + ct) * a.rows + r] = mine;
  }
  if (want_col) {
#pragma unroll
    for (uint32_t q = 0; q < 8; ++q) {
      const uint32_t s = BLOCK_2D ? both : scale_byte(col_max[q]);
      turned[place(8 * cg + q, rg)] = encode_col(v, q, s);
      if (lane < 16) col_bytes[8 * cg + q][wave] = static_cast<uint8_t>(s);
    }
  }
  __syncthreads();

  const uint32_t piece = t % 4;  // 16 bytes of a row of the tile
  const u32x4 *const from[2] = {reinterpret_cast<const u32x4 *>(straight), reinterpret_cast<const u32x4 *>(turned)};
#pragma unroll
  for (uint32_t side = 0; side < 2; ++side) {
    uint8_t *const data = side == 0 ? a.row_data : a.col_data;
    if (data == nullptr) continue;
    const uint32_t n = side == 0 ? a.rows : a.cols, n0 = side == 0 ? r0 : c0, kt = side == 0 ? ct : rt;
    const uint64_t pitch = static_cast<uint64_t>(side == 0 ? a.col_tiles : a.row_tiles) * (kTile / 2);
    uint8_t *const dst = data + (static_cast<uint64_t>(batch) * n + n0) * pitch + kt * (kTile / 2) + 16 * piece;
#pragma unroll
    for (uint32_t h = 0; h < 2; ++h) {
      const uint32_t i = t / 4 + 64 * h;
      if (n0 + i < n) put<STREAM>(reinterpret_cast<u32x4 *>(dst + i * pitch), from[side][place(i, 4 * piece) / 4]);
    }
  }
  if (want_col && t < kTile && c0 + t < a.cols)
    a.col_scales[(static_cast<uint64_t>(batch) * a.row_tiles + rt) * a.cols + c0 + t] = *reinterpret_cast<const uint32_t *>(col_bytes[t]);
}

// ---------------------------------------------------------------------------
// The values: y [n][k] of code * X, exact in binary32 and BF16 both. A thread
// makes kUnits pieces of 16 bytes, a workgroup's worth apart, so that a wave's
// stores are contiguous.
// ---------------------------------------------------------------------------
struct BackArgs {
  const uint8_t *data, *scales;
  void *y;
  uint32_t n, k, kblocks;
  uint32_t per_row;  // pieces of a row
  uint64_t units;    // of all rows of all matrices
};
constexpr uint32_t kUnits = 4;

template <bool OUT32>
__global__ __launch_bounds__(kThreads) void k_mxfp4_dequantize(BackArgs a) {
  constexpr uint32_t per = OUT32 ? 4 : 8;  // values of a piece
  const uint64_t unit0 = static_cast<uint64_t>(block_of_long_grid()) * (kUnits * kThreads) + threadIdx.x;
  uint64_t row[kUnits];
  uint32_t at[kUnits], w[kUnits], s[kUnits];
#pragma unroll
  for (uint32_t i = 0; i < kUnits; ++i) {
    const uint64_t unit = min(unit0 + i * kThreads, a.units - 1);  // past the end: the last one again
    // (a division of 32 bits takes a quarter of one of 64)
    row[i] = a.units <= 0xFFFFFFFFu ? static_cast<uint32_t>(unit) / a.per_row : unit / a.per_row;
    at[i] = static_cast<uint32_t>(unit - row[i] * a.per_row) * per;
    const uint32_t batch = a.units <= 0xFFFFFFFFu ? static_cast<uint32_t>(row[i]) / a.n : static_cast<uint32_t>(row[i] / a.n);
    const uint32_t r = static_cast<uint32_t>(row[i] - static_cast<uint64_t>(batch) * a.n);
    const uint8_t *from = a.data + row[i] * (static_cast<uint64_t>(a.kblocks) * (kFp8Block / 2)) + at[i] / 2;
    w[i] = OUT32 ? *reinterpret_cast<const uint16_t *>(from) : *reinterpret_cast<const uint32_t *>(from);
    s[i] = a.scales[((static_cast<uint64_t>(batch) * a.kblocks + at[i] / kFp8Block) * a.n + r) * 4 + at[i] / 32 % 4];
  }
#pragma unroll
  for (uint32_t i = 0; i < kUnits; ++i) {
    if (unit0 + i * kThreads >= a.units) continue;
    // 2^(s - 127), which is subnormal for 0; NaN for 255
    const float x = __uint_as_float(s[i] == 0 ? 0x00400000u : s[i] == 255 ? 0x7FC00000u : s[i] << 23);
    typedef float f2 __attribute__((ext_vector_type(2)));
    float v[per];
    const f2 p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i], 1.0f, 0), p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i], 1.0f, 1);
    v[0] = p0.x * x, v[1] = p0.y * x, v[2] = p1.x * x, v[3] = p1.y * x;
    if constexpr (!OUT32) {
      const f2 p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i], 1.0f, 2), p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[i], 1.0f, 3);
      v[4] = p2.x * x, v[5] = p2.y * x, v[6] = p3.x * x, v[7] = p3.y * x;
    }
    const uint64_t to = row[i] * a.k + at[i];
    if (at[i] + per <= a.k) {
      u32x4_any o;
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = OUT32 ? __float_as_uint(v[e % per]) : bf16_pair(v[2 * e % per], v[(2 * e + 1) % per]);
      if (OUT32) *reinterpret_cast<u32x4_any *>(static_cast<float *>(a.y) + to) = o;
      else *reinterpret_cast<u32x4_any *>(static_cast<uint16_t *>(a.y) + to) = o;
      continue;
    }
#pragma unroll
    for (uint32_t e = 0; e < per; ++e) {
      if (at[i] + e >= a.k) continue;
      if (OUT32) static_cast<float *>(a.y)[to + e] = v[e];
      else static_cast<uint16_t *>(a.y)[to + e] = static_cast<uint16_t>(bf16_pair(v[e], 0.0f));
    }
  }
}

template <int DT, bool BLOCK_2D>
hipError_t launch(const Args &a, hipStream_t s) {
  if (a.tiles == 0) return hipSuccess;
  const uint64_t in = static_cast<uint64_t>(a.tiles) * kTile * kTile * (DT == kBF16 ? 2 : 4);
  if (a.row_slots != nullptr || in < kStreamBelow) hipLaunchKernelGGL((k_mxfp4_quantize<DT, BLOCK_2D, true>), long_grid(a.tiles), dim3(kThreads), 0, s, a);
  else hipLaunchKernelGGL((k_mxfp4_quantize<DT, BLOCK_2D, false>), long_grid(a.tiles), dim3(kThreads), kIdleLds, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mxfp4_quantize(const Mxfp4Quantize &p, int dtype, bool block_2d, hipStream_t s) {
  const uint32_t row_tiles = (p.rows + kTile - 1) / kTile, col_tiles = (p.cols + kTile - 1) / kTile;
  const Args a{p.x, p.rows, p.cols, row_tiles, col_tiles, p.batch * row_tiles * col_tiles, p.row_slots, p.slots, p.topk,
               p.row_data, p.col_data, reinterpret_cast<uint32_t *>(p.row_scales), reinterpret_cast<uint32_t *>(p.col_scales)};
  if (dtype == kBF16) return block_2d ? launch<kBF16, true>(a, s) : launch<kBF16, false>(a, s);
  return block_2d ? launch<kFP32, true>(a, s) : launch<kFP32, false>(a, s);
}

hipError_t launch_mxfp4_dequantize(const uint8_t *data, const uint8_t *scales, uint32_t batch, uint32_t n, uint32_t k, bool out_fp32, void *y,
                                   hipStream_t s) {
  const uint32_t per = out_fp32 ? 4 : 8;
  BackArgs a{data, scales, y, n, k, (k + kFp8Block - 1) / kFp8Block, (k + per - 1) / per, 0};
  a.units = static_cast<uint64_t>(batch) * n * a.per_row;
  const dim3 grid = long_grid((a.units + kUnits * kThreads - 1) / (kUnits * kThreads));
  if (out_fp32) hipLaunchKernelGGL((k_mxfp4_dequantize<true>), grid, dim3(kThreads), 0, s, a);
  else hipLaunchKernelGGL((k_mxfp4_dequantize<false>), grid, dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace nvfp4
