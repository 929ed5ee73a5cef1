// Block-scaled FP8 quantization: E4M3 codes with one binary32 decode scale
// for each block of 128 (1x128 along a row, or 128x128), in the row-wise and
// the column-wise (transposed) orientation from one read of the input.
//
//   s = fl(max|v| / 448)   e = fl(1 / s), at most FLT_MAX; 0 unless s > 0
//   code = E4M3(fl(v * e)), nearest even
//
// No value needs a clamp: |v| <= 448 s (1 + 2^-22) and e <= (1 / s) (1 + 2^-24) for
// s from 2^-128 up (below that FLT_MAX cuts e short, and |v e| < 448), so |v e| exceeds
// 448 by 2^-21 of it at most, and what is below 464 rounds to 448. A block with an infinity
// or a NaN has s infinite or NaN, hence e 0: its finite values get zero codes, the
// others 0 * inf or 0 * NaN, which converts to the NaN code, so that all of it
// decodes to NaN. (A clamp by v_med3_f32 would make -448 of those NaN, and -inf of
// an infinity of either sign.)
//
// One workgroup per 128x128 tile, in registers: thread t holds the 8x8 patch
// at rows 8 (t / 16), columns 8 (t % 16), so that 16 lanes read 256
// contiguous bytes of a BF16 row, each lane's 8 codes of a row are one
// 8-byte store (128 contiguous bytes for the 16 lanes), and the 8 codes that
// it has of a column are one 8-byte word of the transposed tile, which goes
// through LDS so that it leaves by whole rows too. A row's maximum is taken
// across 16 lanes, a column's across the wave and then the four waves; then
// one thread a row (column) divides, and everyone reads the multipliers.
// Bound by HBM: 2 (or 4) bytes read and 1 or 2 written for each value. 32 x
// 2048x4096 BF16 in 2D both ways moves 5.8 TB/s (185 us), where a copy on the
// same card moves 5.0; 8192x5120 1D both ways 5.5 TB/s.
// Columns and rows past the end count as zeros; each orientation's rows are
// padded to a multiple of 128 with zero codes, which every tile writes whole.
#include "codec.h"
#include "launch.h"

namespace nvfp4 {
namespace {

constexpr uint32_t kThreads = 256;
constexpr uint32_t kTile = kFp8Block;
constexpr float kE4m3Max = 448.0f;

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));  // rows start at any element
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// Outputs that the L2s together do not hold are stored past the caches, which
// keep the input instead: 8192x5120 both ways 32.6 -> 30.7 us, 32 x 2048x4096 in 2D
// both ways 214 -> 204 us, 36864 gathered rows of 5120 columns both ways 152 -> 127 us.
// (Column-wise alone that costs time, 118 -> 131 us at 36864x5120, and is not done.)
constexpr uint64_t kL2Bytes = uint64_t{8} * 4 << 20;
// LDS that is asked for and not used, so that a CU takes five workgroups: with
// more, the 2D case above takes 204 us, with five 185 us, with four 191 us.
constexpr uint32_t kSpareLds = 12000;

template <bool STREAM, typename T>
__device__ __forceinline__ void put(T *to, T v) {
  if (STREAM) __builtin_nontemporal_store(v, to);
  else *to = v;
}

struct Args {
  const void *x;
  uint32_t rows, cols;             // of one matrix
  uint32_t row_tiles, col_tiles;
  uint32_t tiles;                  // of all matrices
  const int32_t *row_slots;
  uint32_t slots, topk;
  uint8_t *row_data, *col_data;
  float *row_scales, *col_scales;
};

// Maximum over the 16 lanes of a DPP row.
__device__ __forceinline__ uint32_t row16_max(uint32_t v) {
  v = max(v, dpp_mov<kQuadXor1>(v));
  v = max(v, dpp_mov<kQuadXor2>(v));
  v = max(v, dpp_mov<0x141>(v));
  return max(v, dpp_mov<0x140>(v));
}

// |v| as its bit pattern: non-negative floats order like integers, and NaN
// is above everything, so a block with a NaN gets a NaN scale.
__device__ __forceinline__ uint32_t mag(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

struct Scale {
  float s, e;
};

__device__ __forceinline__ Scale block_scale_fp8(uint32_t amax_bits) {
  Scale r;
  r.s = __uint_as_float(amax_bits) / kE4m3Max;
  r.e = r.s > 0.0f ? fminf(1.0f / r.s, kFltMax) : 0.0f;
  return r;
}

__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true));
}

// A thread's 8x8 patch. BF16 stays packed, two values a word, until it is
// encoded: half the registers, so twice the workgroups a CU, and the maxima
// are 16-bit ones, two at a time (magnitudes order like their bits in both
// types). word(): columns 2 i and 2 i + 1 of row p.
template <int DT>
struct Patch;

typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t pk_max(uint32_t a, uint32_t b) {
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
}

template <>
struct Patch<kBF16> {
  u32x4 w[8];
  __device__ __forceinline__ void load(int p, const void *x, uint64_t at, uint32_t left) {
    const uint16_t *src = static_cast<const uint16_t *>(x) + at;
    if (left >= 8) {
      w[p] = *reinterpret_cast<const u32x4_any *>(src);
      return;
    }
    uint32_t e[8];
#pragma unroll
    for (uint32_t i = 0; i < 8; ++i) e[i] = i < left ? src[i] : 0u;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[p][i] = e[2 * i] | e[2 * i + 1] << 16;
  }
  __device__ __forceinline__ void clear(int p) { w[p] = u32x4{0, 0, 0, 0}; }
  __device__ __forceinline__ float get(int p, int q) const { return q & 1 ? bf16_hi(w[p][q / 2]) : bf16_lo(w[p][q / 2]); }
  __device__ __forceinline__ uint32_t masked(int p, int i) const { return w[p][i] & 0x7FFF7FFFu; }
  // largest magnitude of the patch's row p, as the bits of a float
  __device__ __forceinline__ uint32_t row_max(int p) const {
    const uint32_t m = pk_max(pk_max(masked(p, 0), masked(p, 1)), pk_max(masked(p, 2), masked(p, 3)));
    return max(m << 16, m & 0xFFFF0000u);
  }
  // the same of each column, across the four row groups of the wave
  __device__ __forceinline__ void col_max(uint32_t *m) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t v = masked(0, i);
#pragma unroll
      for (int p = 1; p < 8; ++p) v = pk_max(v, masked(p, i));
      v = pk_max(v, static_cast<uint32_t>(__shfl_xor(static_cast<int>(v), 16)));
      v = pk_max(v, static_cast<uint32_t>(__shfl_xor(static_cast<int>(v), 32)));
      m[2 * i] = v << 16;
      m[2 * i + 1] = v & 0xFFFF0000u;
    }
  }
};

template <>
struct Patch<kFP32> {
  float v[8][8];
  __device__ __forceinline__ void load(int p, const void *x, uint64_t at, uint32_t left) {
    const float *src = static_cast<const float *>(x) + at;
    if (left >= 8) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const u32x4_any w = *reinterpret_cast<const u32x4_any *>(src + 4 * h);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[p][4 * h + i] = __uint_as_float(w[i]);
      }
      return;
    }
#pragma unroll
    for (uint32_t i = 0; i < 8; ++i) v[p][i] = i < left ? src[i] : 0.0f;
  }
  __device__ __forceinline__ void clear(int p) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[p][i] = 0.0f;
  }
  __device__ __forceinline__ float get(int p, int q) const { return v[p][q]; }
  __device__ __forceinline__ uint32_t row_max(int p) const {
    uint32_t m = mag(v[p][0]);
#pragma unroll
    for (int q = 1; q < 8; ++q) m = max(m, mag(v[p][q]));
    return m;
  }
  __device__ __forceinline__ void col_max(uint32_t *m) const {
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      m[q] = mag(v[0][q]);
#pragma unroll
      for (int p = 1; p < 8; ++p) m[q] = max(m[q], mag(v[p][q]));
      m[q] = max(m[q], static_cast<uint32_t>(__shfl_xor(static_cast<int>(m[q]), 16)));
      m[q] = max(m[q], static_cast<uint32_t>(__shfl_xor(static_cast<int>(m[q]), 32)));
    }
  }
};

template <int DT, bool BLOCK_2D, bool STREAM>
__global__ __launch_bounds__(kThreads) void k_fp8_quantize(Args a) {
  __shared__ uint32_t row_max[kTile], col_max[kThreads / 64][kTile];
  __shared__ float row_mult[kTile], col_mult[kTile];
  __shared__ u32x2 turned[kTile][16];  // the transposed tile's codes, 8 bytes apiece, see below
  const uint32_t t = threadIdx.x, cg = t % 16, rg = t / 16, lane = t % 64, wave = t / 64;
  const uint32_t block = block_of_long_grid();
  if (block >= a.tiles) return;
  const uint32_t per_batch = a.row_tiles * a.col_tiles, batch = block / per_batch, id = block - batch * per_batch;
  uint32_t ct = id % a.col_tiles, rt = id / a.col_tiles;
  if (a.row_slots != nullptr) {
    // a token's row is read topk times: an XCD (workgroups go to the eight in
    // turn) takes whole strips of 128 columns, so that its L2 keeps them
    const uint32_t strip = id / (8 * a.row_tiles) * 8, in = id - strip * a.row_tiles, wide = min(8u, a.col_tiles - strip);
    ct = strip + in % wide;
    rt = in / wide;
  }
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

  const bool want_col = a.col_data != nullptr;
#pragma unroll
  for (uint32_t p = 0; p < 8; ++p) {
    const uint32_t m = row16_max(v.row_max(p));
    if (cg == 0) row_max[8 * rg + p] = m;
  }
  if (!BLOCK_2D && want_col) {
    uint32_t m[8];
    v.col_max(m);
    if (lane < 16) {
#pragma unroll
      for (int q = 0; q < 8; ++q) col_max[wave][8 * cg + q] = m[q];
    }
  }
  __syncthreads();

  Scale tile_scale{};
  if (BLOCK_2D) {
    tile_scale = block_scale_fp8(wave_max(max(row_max[lane], row_max[lane + 64])));
    if (t == 0) {
      const uint64_t per = static_cast<uint64_t>(a.row_tiles) * a.col_tiles;
      if (a.row_data) a.row_scales[batch * per + static_cast<uint64_t>(ct) * a.row_tiles + rt] = tile_scale.s;
      if (want_col) a.col_scales[batch * per + static_cast<uint64_t>(rt) * a.col_tiles + ct] = tile_scale.s;
    }
  } else {
    if (t < kTile) {
      const Scale s = block_scale_fp8(row_max[t]);
      row_mult[t] = s.e;
      if (a.row_data && r0 + t < a.rows)
        a.row_scales[(static_cast<uint64_t>(batch) * a.col_tiles + ct) * a.rows + r0 + t] = s.s;
    } else if (want_col) {
      const uint32_t i = t - kTile;
      const Scale s = block_scale_fp8(max(max(col_max[0][i], col_max[1][i]), max(col_max[2][i], col_max[3][i])));
      col_mult[i] = s.e;
      if (c0 + i < a.cols) a.col_scales[(static_cast<uint64_t>(batch) * a.row_tiles + rt) * a.cols + c0 + i] = s.s;
    }
    __syncthreads();
  }

  if (a.row_data) {
    uint8_t *dst = a.row_data + static_cast<uint64_t>(batch) * a.rows * (static_cast<uint64_t>(a.col_tiles) * kTile) + c;
#pragma unroll
    for (uint32_t p = 0; p < 8; ++p) {
      const uint32_t r = r0 + 8 * rg + p;
      const float e = BLOCK_2D ? tile_scale.e : row_mult[8 * rg + p];
      u32x2 w;
      w.x = pack4(v.get(p, 0) * e, v.get(p, 1) * e, v.get(p, 2) * e, v.get(p, 3) * e);
      w.y = pack4(v.get(p, 4) * e, v.get(p, 5) * e, v.get(p, 6) * e, v.get(p, 7) * e);
      if (r < a.rows) put<STREAM>(reinterpret_cast<u32x2 *>(dst + static_cast<uint64_t>(r) * (static_cast<uint64_t>(a.col_tiles) * kTile)), w);
    }
  }
  if (want_col) {
    // word (column, row group) sits at slot (row group ^ column / 8): a wave
    // writes four row groups of 16 column groups, which that spreads evenly
    // over the banks, where the plain order would meet on four words
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const float e = BLOCK_2D ? tile_scale.e : col_mult[8 * cg + q];
      u32x2 w;
      w.x = pack4(v.get(0, q) * e, v.get(1, q) * e, v.get(2, q) * e, v.get(3, q) * e);
      w.y = pack4(v.get(4, q) * e, v.get(5, q) * e, v.get(6, q) * e, v.get(7, q) * e);
      turned[8 * cg + q][rg ^ cg] = w;
    }
    __syncthreads();
    const uint64_t pitch = static_cast<uint64_t>(a.row_tiles) * kTile;
    uint8_t *dst = a.col_data + static_cast<uint64_t>(batch) * a.cols * pitch + r0;
#pragma unroll
    for (uint32_t k = 0; k < 4; ++k) {
      const uint32_t i = t / 8 + 32 * k, piece = t % 8;  // column i of the tile, its rows 16 piece ..
      const u32x2 lo = turned[i][(2 * piece) ^ (i / 8)], hi = turned[i][(2 * piece + 1) ^ (i / 8)];
      if (c0 + i < a.cols) put<STREAM>(reinterpret_cast<u32x4 *>(dst + (c0 + i) * pitch + 16 * piece), u32x4{lo.x, lo.y, hi.x, hi.y});
    }
  }
}

}  // namespace

namespace {

template <int DT, bool BLOCK_2D>
hipError_t launch(const Args &a, hipStream_t s) {
  if (a.tiles == 0) return hipSuccess;
  const uint64_t out = static_cast<uint64_t>(a.tiles) * kTile * kTile * ((a.row_data != nullptr) + (a.col_data != nullptr));
  const dim3 grid = long_grid(a.tiles);
  if (out > kL2Bytes && a.row_data != nullptr) hipLaunchKernelGGL((k_fp8_quantize<DT, BLOCK_2D, true>), grid, dim3(kThreads), kSpareLds, s, a);
  else hipLaunchKernelGGL((k_fp8_quantize<DT, BLOCK_2D, false>), grid, dim3(kThreads), kSpareLds, s, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_fp8_quantize(const Fp8Quantize &p, int dtype, bool block_2d, hipStream_t s) {
  const uint32_t row_tiles = (p.rows + kTile - 1) / kTile, col_tiles = (p.cols + kTile - 1) / kTile;
  const Args a{p.x, p.rows, p.cols, row_tiles, col_tiles, p.batch * row_tiles * col_tiles, p.row_slots, p.slots, p.topk,
               p.row_data, p.col_data, p.row_scales, p.col_scales};
  if (dtype == kBF16) return block_2d ? launch<kBF16, true>(a, s) : launch<kBF16, false>(a, s);
  return block_2d ? launch<kFP32, true>(a, s) : launch<kFP32, false>(a, s);
}

}  // namespace nvfp4
