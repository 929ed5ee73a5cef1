// Block-scaled FP8 quantization: E4M3 codes with one binary32 decode scale
// for each block of 128 (1x128 along a row, or 128x128), in the row-wise and
// the column-wise (transposed) orientation from one read of the input.
//
//   s = fl(max|v| / 448)   e = fl(1 / s), 0 when s == 0, at most FLT_MAX
//   code = E4M3(clamp(fl(v * e), -448, 448)), nearest even
//
// One workgroup per 128x128 tile, in registers: thread t holds the 8x8 patch
// at rows 8 (t / 16), columns 8 (t % 16), so that 16 lanes read 256
// contiguous bytes of a BF16 row, each lane's 8 codes of a row are one
// 8-byte store (128 contiguous bytes for the 16 lanes), and the 8 codes that
// it has of a column are one 8-byte word of the transposed tile, which goes
// through LDS so that it leaves by whole rows too. A row's maximum is taken
// across 16 lanes, a column's across the wave and then the four waves; then
// one thread a row (column) divides, and everyone reads the multipliers.
// Bound by HBM: 2 (or 4) bytes read and 1 or 2 written for each value.
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

struct Args {
  const void *x;
  uint32_t rows, cols;             // of one matrix
  uint32_t row_tiles, col_tiles;
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

__device__ __forceinline__ float scaled(float v, float e) { return __builtin_amdgcn_fmed3f(v * e, -kE4m3Max, kE4m3Max); }

__device__ __forceinline__ uint32_t pack4(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return static_cast<uint32_t>(__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true));
}

template <int DT>
__device__ __forceinline__ void load8(const void *x, uint64_t at, uint32_t left, float *v) {
  if (DT == kBF16) {
    const uint16_t *p = static_cast<const uint16_t *>(x) + at;
    if (left >= 8) {
      const u32x4_any w = *reinterpret_cast<const u32x4_any *>(p);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = bf16_lo(w[i]);
        v[2 * i + 1] = bf16_hi(w[i]);
      }
      return;
    }
#pragma unroll
    for (uint32_t i = 0; i < 8; ++i) v[i] = i < left ? __uint_as_float(static_cast<uint32_t>(p[i]) << 16) : 0.0f;
  } else {
    const float *p = static_cast<const float *>(x) + at;
    if (left >= 8) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const u32x4_any w = *reinterpret_cast<const u32x4_any *>(p + 4 * h);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[4 * h + i] = __uint_as_float(w[i]);
      }
      return;
    }
#pragma unroll
    for (uint32_t i = 0; i < 8; ++i) v[i] = i < left ? p[i] : 0.0f;
  }
}

template <int DT, bool BLOCK_2D>
__global__ __launch_bounds__(kThreads) void k_fp8_quantize(Args a) {
  __shared__ uint32_t row_max[kTile], col_max[kThreads / 64][kTile];
  __shared__ float row_mult[kTile], col_mult[kTile];
  __shared__ u32x2 turned[kTile][16];  // the transposed tile's codes, 8 bytes apiece, see below
  const uint32_t t = threadIdx.x, cg = t % 16, rg = t / 16, lane = t % 64, wave = t / 64;
  const uint32_t ct = blockIdx.x % a.col_tiles, rest = blockIdx.x / a.col_tiles;
  const uint32_t rt = rest % a.row_tiles, batch = rest / a.row_tiles;
  const uint32_t r0 = rt * kTile, c0 = ct * kTile;
  const uint32_t c = c0 + 8 * cg;
  const uint32_t left = c < a.cols ? a.cols - c : 0;

  float v[8][8];
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
    if (have) {
      load8<DT>(a.x, src * a.cols + c, left, v[p]);
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q) v[p][q] = 0.0f;
    }
  }

  const bool want_col = a.col_data != nullptr;
#pragma unroll
  for (uint32_t p = 0; p < 8; ++p) {
    uint32_t m = 0;
#pragma unroll
    for (int q = 0; q < 8; ++q) m = max(m, mag(v[p][q]));
    m = row16_max(m);
    if (cg == 0) row_max[8 * rg + p] = m;
  }
  if (!BLOCK_2D && want_col) {
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      uint32_t m = 0;
#pragma unroll
      for (int p = 0; p < 8; ++p) m = max(m, mag(v[p][q]));
      m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 16)));
      m = max(m, static_cast<uint32_t>(__shfl_xor(static_cast<int>(m), 32)));
      if (lane < 16) col_max[wave][8 * cg + q] = m;
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
      w.x = pack4(scaled(v[p][0], e), scaled(v[p][1], e), scaled(v[p][2], e), scaled(v[p][3], e));
      w.y = pack4(scaled(v[p][4], e), scaled(v[p][5], e), scaled(v[p][6], e), scaled(v[p][7], e));
      if (r < a.rows) *reinterpret_cast<u32x2 *>(dst + static_cast<uint64_t>(r) * (static_cast<uint64_t>(a.col_tiles) * kTile)) = w;
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
      w.x = pack4(scaled(v[0][q], e), scaled(v[1][q], e), scaled(v[2][q], e), scaled(v[3][q], e));
      w.y = pack4(scaled(v[4][q], e), scaled(v[5][q], e), scaled(v[6][q], e), scaled(v[7][q], e));
      turned[8 * cg + q][rg ^ cg] = w;
    }
    __syncthreads();
    const uint64_t pitch = static_cast<uint64_t>(a.row_tiles) * kTile;
    uint8_t *dst = a.col_data + static_cast<uint64_t>(batch) * a.cols * pitch + r0;
#pragma unroll
    for (uint32_t k = 0; k < 4; ++k) {
      const uint32_t i = t / 8 + 32 * k, piece = t % 8;  // column i of the tile, its rows 16 piece ..
      const u32x2 lo = turned[i][(2 * piece) ^ (i / 8)], hi = turned[i][(2 * piece + 1) ^ (i / 8)];
      if (c0 + i < a.cols) *reinterpret_cast<u32x4 *>(dst + (c0 + i) * pitch + 16 * piece) = u32x4{lo.x, lo.y, hi.x, hi.y};
    }
  }
}

}  // namespace

hipError_t launch_fp8_quantize(const Fp8Quantize &p, int dtype, bool block_2d, hipStream_t s) {
  Args a{p.x, p.rows, p.cols, (p.rows + kTile - 1) / kTile, (p.cols + kTile - 1) / kTile, p.row_slots, p.slots, p.topk,
         p.row_data, p.col_data, p.row_scales, p.col_scales};
  const uint64_t blocks = static_cast<uint64_t>(p.batch) * a.row_tiles * a.col_tiles;
  if (blocks == 0) return hipSuccess;
  const dim3 grid(static_cast<uint32_t>(blocks));
  if (dtype == kBF16) {
    if (block_2d) hipLaunchKernelGGL((k_fp8_quantize<kBF16, true>), grid, dim3(kThreads), 0, s, a);
    else hipLaunchKernelGGL((k_fp8_quantize<kBF16, false>), grid, dim3(kThreads), 0, s, a);
  } else {
    if (block_2d) hipLaunchKernelGGL((k_fp8_quantize<kFP32, true>), grid, dim3(kThreads), 0, s, a);
    else hipLaunchKernelGGL((k_fp8_quantize<kFP32, false>), grid, dim3(kThreads), 0, s, a);
  }
  return hipGetLastError();
}

}  // namespace nvfp4
