// The 8x8 patch of a tile that a thread of a quantize kernel holds, and what
// its maxima and stores are made of.
#pragma once

#include "codec.h"
#include "launch.h"

namespace nvfp4 {
namespace {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));  // rows start at any element
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

template <bool STREAM, typename T>
__device__ __forceinline__ void put(T *to, T v) {
  if (STREAM) __builtin_nontemporal_store(v, to);
  else *to = v;
}

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

}  // namespace
}  // namespace nvfp4
