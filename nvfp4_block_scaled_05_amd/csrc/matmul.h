// What the product kernels share: which rows and columns a workgroup takes, loads
// straight to LDS, and stores of rows that start at any element.
#pragma once

#include "codec.h"
#include "launch.h"

namespace nvfp4 {
namespace {

constexpr uint32_t kWave = 64;

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_any __attribute__((ext_vector_type(4), aligned(2)));  // rows of d start at any element

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
__device__ __forceinline__ Part find_rows(const int32_t *offsets, uint32_t groups, uint32_t m, uint32_t kblocks, uint32_t tile) {
  const uint32_t lane = threadIdx.x % kWave;
  uint32_t start[5], tiles[4], sum = 0;
#pragma unroll
  for (uint32_t i = 0; i < 5; ++i) start[i] = clamped(offsets[min(4 * lane + i, groups)], m);
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
  Part r{0, 0, 0, kblocks, 0, false};
  if (past == 0) {
    const uint32_t total = __builtin_amdgcn_readlane(scan, kWave - 1);
    const uint64_t m0 = clamped(offsets[groups], m) + static_cast<uint64_t>(tile - total) * BM;
    r.m0 = static_cast<uint32_t>(min(m0, static_cast<uint64_t>(m)));
    r.m_end = m;
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
__device__ __forceinline__ void tile_of(uint32_t id, uint32_t tiles_n, uint32_t &tm, uint32_t &tn) {
  const uint32_t total = gridDim.x;
  if (id < total / (kXcds * kRun) * (kXcds * kRun)) {
    const uint32_t in = id % (kXcds * kRun);
    id = id - in + in % kXcds * kRun + in / kXcds;
  }
  const uint32_t rows = total / tiles_n, band = id / (kPatch * tiles_n), in = id - band * kPatch * tiles_n;
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

}  // namespace
}  // namespace nvfp4
