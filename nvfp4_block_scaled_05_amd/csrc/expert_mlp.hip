// A whole expert layer for a few tokens, in two launches:
//
//   h[s] = act(w1[e] x[t])            for each slot s = t topk + j with expert e = ids[t][j]
//   out[t] = sum over j of weights[t][j] w2[e] h[s]
//
// act(g, u) = silu(g) u for the two halves of w1's rows, or silu(g); weights in
// MXFP4 or block-scaled FP8 (128x128 blocks), x and out BF16. Bound by reading
// the weights of the experts in use, once each; so the codes are widened to BF16
// in registers (exact: E2M1 values times a power of two, and E4M3 values, are
// BF16 values) and multiplied by v_mfma_f32_16x16x32_bf16, which sums to binary32,
// and no activation is quantized. h is rounded to BF16 on its way to the second
// kernel, which reads all of it in every workgroup: half the bytes and
// products of FP32, for an error below that of out's own rounding.
//
// A wave's fragment of a block of 128 along k is 16 rows of weights: lane l has
// 32 values of row l % 16, and of token l % 16's row the same 32, so which
// values those are is free. The first operand is the tokens, the second the
// weights: lane l ends with tokens 4 (l / 16) .. + 3 of row l % 16.
#include "codec.h"
#include "launch.h"
#include "matmul.h"

namespace nvfp4 {
namespace {

constexpr uint32_t kBlock = kFp8Block;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// What lane l holds of a row's block and of a token's, and what the block's sum is scaled by.
struct Mx {
  static constexpr uint32_t kRowBytes = kBlock / 2, kUnroll = 8;
  typedef uint32_t Scale;  // the row's word of four bytes
  struct Raw {
    u32x4 w;
  };
  // bytes 16 q .. of the row: values 32 q ..
  static __device__ __forceinline__ Raw load(const uint8_t *row, uint32_t q) { return {*reinterpret_cast<const u32x4 *>(row + 16 * q)}; }
  // the scales of rows 0 .. of a matrix: row r's of block kb
  static __device__ __forceinline__ Scale scale(const void *scales, uint32_t n, uint32_t kb, uint32_t r) {
    return static_cast<const uint32_t *>(scales)[static_cast<uint64_t>(kb) * n + r];
  }
  static __host__ __device__ uint64_t scale_bytes(uint32_t n, uint32_t kblocks) { return static_cast<uint64_t>(n) * kblocks * 4; }
  // value of the token's row that piece p (0 .. 3) of 8 begins at
  static __device__ __forceinline__ uint32_t at(uint32_t q, uint32_t p) { return 32 * q + 8 * p; }
  static __device__ __forceinline__ void widen(const Raw &r, Scale s, uint32_t q, bf16x8 *f) {
    const uint32_t byte = s >> (8 * q) & 255;
    const float x = __uint_as_float(byte == 255 ? 0x7FC00000u : byte == 0 ? 0x00400000u : byte << 23);
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(r.w[p], x, 0), b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(r.w[p], x, 1);
      const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(r.w[p], x, 2), d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(r.w[p], x, 3);
      f[p] = bf16x8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
    }
  }
  static __device__ __forceinline__ f32x4 add(f32x4 acc, const bf16x8 *t, const bf16x8 *w, Scale) {
#pragma unroll
    for (int p = 0; p < 4; ++p) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(t[p], w[p], acc, 0, 0, 0);
    return acc;
  }
};

struct F8 {
  static constexpr uint32_t kRowBytes = kBlock, kUnroll = 4;
  typedef float Scale;
  struct Raw {
    u32x4 w[2];
  };
  // bytes 16 q .. and 64 + 16 q .. of the row, so that four lanes read 64 contiguous bytes
  static __device__ __forceinline__ Raw load(const uint8_t *row, uint32_t q) {
    return {{*reinterpret_cast<const u32x4 *>(row + 16 * q), *reinterpret_cast<const u32x4 *>(row + 64 + 16 * q)}};
  }
  static __device__ __forceinline__ Scale scale(const void *scales, uint32_t n, uint32_t kb, uint32_t r) {
    return static_cast<const float *>(scales)[static_cast<uint64_t>(kb) * ((n + kBlock - 1) / kBlock) + r / kBlock];
  }
  static __host__ __device__ uint64_t scale_bytes(uint32_t n, uint32_t kblocks) { return static_cast<uint64_t>((n + kBlock - 1) / kBlock) * kblocks * 4; }
  static __device__ __forceinline__ uint32_t at(uint32_t q, uint32_t p) { return p / 2 * 64 + 16 * q + p % 2 * 8; }
  static __device__ __forceinline__ void widen(const Raw &r, Scale, uint32_t, bf16x8 *f) {
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const uint32_t x = r.w[p / 2][p % 2 * 2], y = r.w[p / 2][p % 2 * 2 + 1];
      const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x, 1.0f, false), b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x, 1.0f, true);
      const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(y, 1.0f, false), d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(y, 1.0f, true);
      f[p] = bf16x8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
    }
  }
  static __device__ __forceinline__ f32x4 add(f32x4 acc, const bf16x8 *t, const bf16x8 *w, Scale s) {
    f32x4 c{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int p = 0; p < 4; ++p) c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(t[p], w[p], c, 0, 0, 0);
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] = __builtin_fmaf(c[e], s, acc[e]);
    return acc;
  }
};

// The workspace: words[0] the number of experts in use; from words[1] on kMaxGroups entries
// of (expert, first place in the list, slots); then the list of slots, expert after
// expert, each expert's in order; then h [slots][pitch] at kHidden.
constexpr uint32_t kEntry = 3, kList = 4 + kEntry * kMaxGroups, kHidden = (kList + kMlpMaxSlots) * 4;
static_assert(kHidden % 16 == 0 && kHidden == kMlpHeader, "h is aligned");

struct Args {
  const uint16_t *x;
  const void *ids;
  uint32_t wide;  // 64-bit ids
  const float *weights;
  const uint8_t *w1, *w2;
  const void *s1, *s2;
  uint32_t *workspace;
  uint16_t *out;
  uint32_t tokens, topk, slots, experts;
  uint32_t cols, hidden, kblocks1, kblocks2;
  uint32_t strips;  // of the first kernel's rows
};

__device__ __forceinline__ uint32_t id_of(const Args &p, uint32_t slot) {
  // an id that is none counts as the expert past the last one
  const int64_t id = p.wide ? static_cast<const int64_t *>(p.ids)[slot] : static_cast<const int32_t *>(p.ids)[slot];
  return id < 0 || id >= p.experts ? p.experts : static_cast<uint32_t>(id);
}

// Eight values of a row of x from `at` on, zeros from `cols` on.
__device__ __forceinline__ bf16x8 tokens8(const uint16_t *row, uint32_t at, uint32_t cols) {
  if (at + 8 <= cols) return __builtin_bit_cast(bf16x8, *reinterpret_cast<const u32x4_any *>(row + at));
  uint32_t e[8];
#pragma unroll
  for (uint32_t i = 0; i < 8; ++i) e[i] = at + i < cols ? row[at + i] : 0u;
  return __builtin_bit_cast(bf16x8, u32x4{e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16});
}

__device__ __forceinline__ float silu(float v) { return v / (1.0f + __expf(-v)); }

// ---------------------------------------------------------------------------
// h: a workgroup takes one expert and 16 units of h (32 where w1 has no second
// half), the blocks along k dealt out to its KS waves, whose sums meet in LDS.
// It finds its expert, the blockIdx-th of those in use, and the expert's
// slots from the ids by itself; the workgroups of the first strip write the
// lists down for the second kernel.
// ---------------------------------------------------------------------------
template <typename F, uint32_t KS, uint32_t MT, uint32_t U, bool GATED>
__device__ __forceinline__ void hidden_tile(const Args &p, uint32_t expert, uint32_t unit0, const uint32_t *list, uint32_t count,
                                            f32x4 (*red)[2][4][kWave]) {
  const uint32_t lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const uint32_t i16 = lane % 16, q = lane / 16;
  const uint32_t n = p.hidden * (GATED ? 2 : 1);
  const uint64_t pitch = static_cast<uint64_t>(p.kblocks1) * F::kRowBytes;
  const uint8_t *w = p.w1 + static_cast<uint64_t>(expert) * n * pitch;
  const uint8_t *scales = static_cast<const uint8_t *>(p.s1) + expert * F::scale_bytes(n, p.kblocks1);
  // rows of w1 past h's units repeat its last one, and their results are not used
  uint32_t row[2];
  const uint8_t *from[2];
#pragma unroll
  for (uint32_t t = 0; t < 2; ++t) {
    row[t] = min(unit0 + i16 + (GATED ? 0 : 16 * t), p.hidden - 1) + (GATED ? p.hidden * t : 0);
    from[t] = w + row[t] * pitch;
  }
  const uint16_t *x[MT];
#pragma unroll
  for (uint32_t i = 0; i < MT; ++i) x[i] = p.x + static_cast<uint64_t>(list[min(16 * i + i16, count - 1)] / p.topk) * p.cols;

  f32x4 acc[MT][2];
#pragma unroll
  for (uint32_t i = 0; i < MT; ++i) acc[i][0] = acc[i][1] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
  for (uint32_t kb0 = wave; kb0 < p.kblocks1; kb0 += U * KS) {
    typename F::Raw raw[U][2];
    typename F::Scale s[U][2];
    bf16x8 tok[U][MT][4];
#pragma unroll
    for (uint32_t u = 0; u < U; ++u) {
      const uint32_t kb = min(kb0 + u * KS, p.kblocks1 - 1);  // past the end: loaded again, not used
#pragma unroll
      for (uint32_t t = 0; t < 2; ++t) {
        raw[u][t] = F::load(from[t] + static_cast<uint64_t>(kb) * F::kRowBytes, q);
        s[u][t] = F::scale(scales, n, kb, row[t]);
      }
#pragma unroll
      for (uint32_t i = 0; i < MT; ++i)
#pragma unroll
        for (uint32_t e = 0; e < 4; ++e) tok[u][i][e] = tokens8(x[i], kb * kBlock + F::at(q, e), p.cols);
    }
#pragma unroll
    for (uint32_t u = 0; u < U; ++u) {
      if (kb0 + u * KS >= p.kblocks1) break;
#pragma unroll
      for (uint32_t t = 0; t < 2; ++t) {
        bf16x8 f[4];
        F::widen(raw[u][t], s[u][t], q, f);
#pragma unroll
        for (uint32_t i = 0; i < MT; ++i) acc[i][t] = F::add(acc[i][t], tok[u][i], f, s[u][t]);
      }
    }
  }
#pragma unroll
  for (uint32_t i = 0; i < MT; ++i)
#pragma unroll
    for (uint32_t t = 0; t < 2; ++t) red[wave][t][i][lane] = acc[i][t];
  lds_barrier();
  uint16_t *h = reinterpret_cast<uint16_t *>(reinterpret_cast<uint8_t *>(p.workspace) + kHidden);
  for (uint32_t it = wave; it < (GATED ? MT : 2 * MT); it += KS) {
    const uint32_t i = GATED ? it : it / 2, t = GATED ? 0 : it % 2;
    f32x4 g = red[0][t][i][lane], u{};
#pragma unroll
    for (uint32_t k = 1; k < KS; ++k) g += red[k][t][i][lane];
    if (GATED) {
      u = red[0][1][i][lane];
#pragma unroll
      for (uint32_t k = 1; k < KS; ++k) u += red[k][1][i][lane];
    }
    const uint32_t unit = unit0 + 16 * t + i16;
#pragma unroll
    for (uint32_t e = 0; e < 4; ++e) {
      const uint32_t place = 16 * i + 4 * q + e;
      // units past the last one, up to the block's end, are zeros
      const float v = unit < p.hidden ? (GATED ? silu(g[e]) * u[e] : silu(g[e])) : 0.0f;
      if (place < count && unit < p.kblocks2 * kBlock)
        h[static_cast<uint64_t>(list[place]) * (p.kblocks2 * kBlock) + unit] = static_cast<uint16_t>(bf16_pair(v, 0.0f));
    }
  }
  lds_barrier();
}

template <typename F, uint32_t KS, bool GATED>
__global__ __launch_bounds__(KS *kWave) void k_mlp_hidden(Args p) {
  __shared__ f32x4 red[KS][2][4][kWave];
  __shared__ uint32_t used[kMaxGroups / 32], list[kMlpMaxSlots], found[2];
  const uint32_t t = threadIdx.x, lane = t % kWave;
  const uint32_t strip = blockIdx.x % p.strips, rank = blockIdx.x / p.strips;
  if (t < kMaxGroups / 32) used[t] = 0;
  lds_barrier();
  for (uint32_t s = t; s < p.slots; s += KS * kWave) {
    const uint32_t id = id_of(p, s);
    list[s] = id;  // the ids, for now
    if (id < p.experts) atomicOr(&used[id / 32], 1u << (id % 32));
  }
  lds_barrier();
  uint32_t expert = p.experts, in_use = 0;
#pragma unroll
  for (uint32_t i = 0; i < kMaxGroups / 32; ++i) {
    uint32_t w = used[i];
    const uint32_t n = __popc(w);
    if (rank >= in_use && rank < in_use + n) {
      for (uint32_t skip = rank - in_use; skip > 0; --skip) w &= w - 1;
      expert = 32 * i + static_cast<uint32_t>(__builtin_ctz(w));
    }
    in_use += n;
  }
  expert = __builtin_amdgcn_readfirstlane(expert);
  if (strip == 0 && rank == 0 && t == 0) p.workspace[0] = in_use;
  if (expert == p.experts) return;
  if (t < kWave) {  // one wave puts the expert's slots in order; what it writes is behind what it reads
    uint32_t count = 0, before = 0;
    for (uint32_t s0 = 0; s0 < p.slots; s0 += kWave) {
      const uint32_t id = s0 + lane < p.slots ? list[s0 + lane] : p.experts;
      const uint64_t mine = __ballot(id == expert);
      before += __popcll(__ballot(id < expert));
      if (id == expert) list[count + __popcll(mine & ((uint64_t{1} << lane) - 1))] = s0 + lane;
      count += __popcll(mine);
    }
    if (lane == 0) found[0] = count, found[1] = before;
  }
  lds_barrier();
  const uint32_t count = __builtin_amdgcn_readfirstlane(found[0]);
  if (strip == 0) {
    const uint32_t before = __builtin_amdgcn_readfirstlane(found[1]);
    if (t < kEntry) p.workspace[1 + kEntry * rank + t] = t == 0 ? expert : t == 1 ? before : count;
    for (uint32_t i = t; i < count; i += KS * kWave) p.workspace[kList + before + i] = list[i];
  }
  const uint32_t unit0 = strip * (GATED ? 16 : 32);
  for (uint32_t at = 0; at < count;) {
    const uint32_t left = count - at;
    if (left <= 16) {
      hidden_tile<F, KS, 1, 4, GATED>(p, expert, unit0, list + at, left, red);
      at += 16;
    } else if (left <= 32) {
      hidden_tile<F, KS, 2, 2, GATED>(p, expert, unit0, list + at, left, red);
      at += 32;
    } else {
      hidden_tile<F, KS, 4, 1, GATED>(p, expert, unit0, list + at, min(left, 64u), red);
      at += 64;
    }
  }
}

// ---------------------------------------------------------------------------
// out: a workgroup takes 16 columns. Its waves go through the experts in use,
// each expert by one wave or (few experts) its blocks along k by `parts` of
// them, and leave each slot's product with the expert's 16 rows in LDS, where
// they are added up in the order of the choices: no atomics, and nothing but
// out is written to memory. The next chunk of weights is on its way while one
// is multiplied.
// ---------------------------------------------------------------------------
constexpr uint32_t kOutWaves = 8, kOutCols = 16;
constexpr uint32_t kSums = 1024;  // slots times parts that LDS has room for

template <typename F>
__global__ __launch_bounds__(kOutWaves *kWave) void k_mlp_out(Args p) {
  constexpr uint32_t U = F::kUnroll;
  __shared__ float sums[kSums][kOutCols];
  __shared__ uint32_t table[kList + kMlpMaxSlots];
  const uint32_t lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const uint32_t i16 = lane % 16, q = lane / 16;
  const uint32_t c0 = blockIdx.x * kOutCols;
  for (uint32_t i = threadIdx.x; i < kList + p.slots; i += kOutWaves * kWave) table[i] = p.workspace[i];
  lds_barrier();
  const uint32_t in_use = __builtin_amdgcn_readfirstlane(table[0]);
  const uint32_t *const list = table + kList;

  // parts: as many as there are waves for, chunks of U blocks to deal out, and room in LDS
  const uint32_t chunks_all = (p.kblocks2 + U - 1) / U;
  uint32_t parts = in_use == 0 ? 1 : max(1u, min(min(kOutWaves / in_use, chunks_all), kSums / p.slots));
  const uint32_t per_part = (chunks_all + parts - 1) / parts;
  const uint32_t items = in_use * parts;
  const uint64_t pitch = static_cast<uint64_t>(p.kblocks2) * F::kRowBytes;
  const uint32_t row = min(c0 + i16, p.cols - 1);
  const uint16_t *h = reinterpret_cast<const uint16_t *>(reinterpret_cast<const uint8_t *>(p.workspace) + kHidden);
  const uint32_t h_pitch = p.kblocks2 * kBlock;

  struct Chunk {
    typename F::Raw raw[U];
    typename F::Scale s[U];
  };
  struct Where {
    uint32_t item, pass, chunk;  // pass: of 32 slots of the expert
  };
  auto expert_of = [&](uint32_t item) { return __builtin_amdgcn_readfirstlane(table[1 + kEntry * (item / parts)]); };
  auto count_of = [&](uint32_t item) { return __builtin_amdgcn_readfirstlane(table[1 + kEntry * (item / parts) + 2]); };
  auto chunks_of = [&](uint32_t item) {  // this part's
    const uint32_t first = item % parts * per_part;
    return first >= chunks_all ? 0 : min(per_part, chunks_all - first);
  };
  auto next = [&](Where at) {
    if (++at.chunk < chunks_of(at.item)) return at;
    at.chunk = 0;
    if (32 * ++at.pass < count_of(at.item)) return at;
    at.pass = 0;
    at.item += kOutWaves;
    return at;
  };
  auto load = [&](const Where &at, Chunk &c) {
    const uint32_t expert = expert_of(at.item);
    const uint8_t *from = p.w2 + (static_cast<uint64_t>(expert) * p.cols + row) * pitch;
    const uint8_t *scales = static_cast<const uint8_t *>(p.s2) + expert * F::scale_bytes(p.cols, p.kblocks2);
#pragma unroll
    for (uint32_t u = 0; u < U; ++u) {
      const uint32_t kb = min((at.item % parts * per_part + at.chunk) * U + u, p.kblocks2 - 1);
      c.raw[u] = F::load(from + static_cast<uint64_t>(kb) * F::kRowBytes, q);
      c.s[u] = F::scale(scales, p.cols, kb, row);
    }
  };

  Where at{wave, 0, 0};
  Chunk now, ahead;
  f32x4 acc[2];
  if (at.item < items) load(at, now);
  while (at.item < items) {
    const Where then = next(at);
    if (then.item < items) load(then, ahead);
    const uint32_t first = __builtin_amdgcn_readfirstlane(table[1 + kEntry * (at.item / parts) + 1]) + 32 * at.pass;
    const uint32_t count = min(32u, count_of(at.item) - 32 * at.pass);
    if (at.chunk == 0) acc[0] = acc[1] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const uint32_t kb0 = (at.item % parts * per_part + at.chunk) * U;
    const uint16_t *tok[2];
#pragma unroll
    for (uint32_t i = 0; i < 2; ++i) tok[i] = h + static_cast<uint64_t>(list[first + min(16 * i + i16, count - 1)]) * h_pitch;
    if (chunks_of(at.item) > 0) {
#pragma unroll
      for (uint32_t u = 0; u < U; ++u) {
        if (kb0 + u >= p.kblocks2) break;
        bf16x8 f[4];
        F::widen(now.raw[u], now.s[u], q, f);
#pragma unroll
        for (uint32_t i = 0; i < 2; ++i) {
          if (16 * i >= count) break;
          bf16x8 t[4];
#pragma unroll
          for (uint32_t e = 0; e < 4; ++e) t[e] = *reinterpret_cast<const bf16x8 *>(tok[i] + (kb0 + u) * kBlock + F::at(q, e));
          acc[i] = F::add(acc[i], t, f, now.s[u]);
        }
      }
    }
    if (then.chunk == 0) {  // the pass is done
#pragma unroll
      for (uint32_t i = 0; i < 2; ++i)
#pragma unroll
        for (uint32_t e = 0; e < 4; ++e) {
          const uint32_t place = 16 * i + 4 * q + e;
          if (place < count) sums[at.item % parts * p.slots + list[first + place]][i16] = acc[i][e];
        }
    }
    now = ahead;
    at = then;
  }
  lds_barrier();
  for (uint32_t i = threadIdx.x; i < p.tokens * kOutCols; i += kOutWaves * kWave) {
    const uint32_t t = i / kOutCols, c = i % kOutCols;
    float v = 0.0f;
    for (uint32_t j = 0; j < p.topk; ++j) {
      const uint32_t slot = t * p.topk + j;
      if (id_of(p, slot) == p.experts) continue;
      float y = 0.0f;
      for (uint32_t k = 0; k < parts; ++k) y += sums[k * p.slots + slot][c];
      v += p.weights[slot] * y;
    }
    if (c0 + c < p.cols) p.out[static_cast<uint64_t>(t) * p.cols + c0 + c] = static_cast<uint16_t>(bf16_pair(v, 0.0f));
  }
}

template <typename F, uint32_t KS>
hipError_t launch_hidden(const Args &a, bool gated, hipStream_t s) {
  const uint64_t blocks = static_cast<uint64_t>(a.strips) * min(a.experts, a.slots);
  if (blocks * KS * kWave >= kMaxThreads1D) return hipErrorInvalidConfiguration;
  if (gated) hipLaunchKernelGGL((k_mlp_hidden<F, KS, true>), dim3(static_cast<uint32_t>(blocks)), dim3(KS * kWave), 0, s, a);
  else hipLaunchKernelGGL((k_mlp_hidden<F, KS, false>), dim3(static_cast<uint32_t>(blocks)), dim3(KS * kWave), 0, s, a);
  return hipGetLastError();
}

template <typename F>
hipError_t launch(const Args &a, bool gated, hipStream_t s) {
  const hipError_t e = a.kblocks1 >= 8 ? launch_hidden<F, 8>(a, gated, s) : launch_hidden<F, 2>(a, gated, s);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((k_mlp_out<F>), dim3((a.cols + kOutCols - 1) / kOutCols), dim3(kOutWaves * kWave), 0, s, a);
  return hipGetLastError();
}

}  // namespace

uint64_t expert_mlp_workspace_bytes(uint64_t slots, uint64_t hidden) {
  return kHidden + slots * ((hidden + kBlock - 1) / kBlock * kBlock) * 2;
}

hipError_t launch_expert_mlp(const ExpertMlp &p, hipStream_t s) {
  Args a{static_cast<const uint16_t *>(p.x), p.ids, p.wide, p.weights, p.w1, p.w2, p.s1, p.s2, p.workspace, static_cast<uint16_t *>(p.out),
         p.tokens, p.topk, p.tokens * p.topk, p.experts, p.cols, p.hidden, (p.cols + kBlock - 1) / kBlock, (p.hidden + kBlock - 1) / kBlock, 0};
  // units up to the end of the last block, so that what the second kernel reads of h is written
  const uint32_t units = a.kblocks2 * kBlock, each = p.gated ? 16 : 32;
  a.strips = (units + each - 1) / each;
  return p.fp8 ? launch<F8>(a, p.gated, s) : launch<Mx>(a, p.gated, s);
}

}  // namespace nvfp4
