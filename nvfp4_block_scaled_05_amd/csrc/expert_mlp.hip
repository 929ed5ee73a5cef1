// A whole expert layer for a few tokens, in three launches:
//
//   h[s] = act(w1[e] x[t])            for each slot s = t topk + j with expert e = ids[t][j]
//   y[s] = w2[e] h[s]
//   out[t] = sum over j of weights[t][j] y[s]
//
// act(g, u) = silu(g) u for the two halves of w1's rows, or silu(g); weights in
// MXFP4 or block-scaled FP8 (128x128 blocks), x and out BF16. Bound by reading
// the weights of the experts in use, once each up to the 16 or 32 slots an expert
// that a pass takes (and from the L2s again for each further pass); so the codes
// are widened to BF16 in registers (exact: E2M1 and E4M3 values times a power of
// two are BF16 values, but for powers at the ends of the range, see Mx and F8) and
// multiplied by v_mfma_f32_16x16x32_bf16, which sums to binary32, and no
// activation is quantized. h goes from the first kernel to the second as two BF16
// numbers, its rounding and the rest's, 16 bits of mantissa together: with one, out
// is 1.4 times as far off (2.4e-3 in the 2-norm, of which out's own rounding makes
// 1.7e-3). y is FP32.
//
// A wave's fragment of a block of 128 along k is 16 rows of weights: lane l has
// 32 values of row l % 16, and of token l % 16's row the same 32, so which
// values those are is free. The first operand is the tokens, the second the
// weights: lane l ends with tokens 4 (l / 16) .. + 3 of row l % 16.
//
// Both products run in the same form: one workgroup a CU, which takes a run of
// tasks, each 16 NT rows of one expert's weights (gated: two rows for each of 8 NT
// units) for up to 16 MT of its tokens, the blocks along k dealt out to eight waves
// (or, where rows are short, to fewer, beside others with rows of their own),
// whose sums meet in LDS: late in the next task, since at a task's own end
// the waves waited for each other (64 tokens, 61 experts of 2 x 2048 x 4096: 141 -> 137 us
// for the first product, 80 -> 76 for the second). The tokens' rows stay in registers
// from task to task (where k fits them), and each register of weights is asked
// for again, for the next task, as soon as it is widened. A row's blocks are
// asked for one after the other, since a line of 128 bytes holds two: 143 -> 123
// us and 80 -> 70.
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
  static constexpr uint32_t kRowBytes = kBlock / 2;
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
  static __device__ __forceinline__ void widen(const Raw &r, Scale s, uint32_t q, bf16x8 *f) { widen_by(r, min(byte_of(s, q), kMostByte), f); }
  // the conversion takes its scale's exponent field as the byte: 0 is 2^-127, 255 NaN
  static __device__ __forceinline__ void widen_by(const Raw &r, uint32_t byte, bf16x8 *f) {
    const float x = __uint_as_float(byte << 23);
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(r.w[p], x, 0), b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(r.w[p], x, 1);
      const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(r.w[p], x, 2), d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(r.w[p], x, 3);
      f[p] = bf16x8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
    }
  }
  static __device__ __forceinline__ uint32_t byte_of(Scale s, uint32_t q) { return s >> (8 * q) & 255; }
  // Under scales 253 and 254 the larger codes are past BF16's range, where an infinity would be wrong, and no number times a zero of
  // x or h: all are widened under 252 at most, and rows with a larger byte (255, which is NaN, among them) are summed again, at the
  // kernel's end. (Within the loop that cost calls that never come there up to 2% of their time, 128 tokens for 8 experts of
  // 2 x 2048 x 4096 108.5 -> 111 us, beside each fragment's products 114: scalar registers run out.)
  static constexpr bool kSumsAgain = true;
  static constexpr uint32_t kMostByte = 252;
  static __device__ __forceinline__ void watch(uint32_t &most, Scale s, uint32_t q) { most = max(most, byte_of(s, q)); }
  static __device__ __forceinline__ bool row_lacks(const void *scales, uint32_t n, uint32_t kblocks, uint32_t r) {
    uint32_t most = 0;
    for (uint32_t piece = 0; piece < kblocks * 4; ++piece) most = max(most, byte_of(scale(scales, n, piece / 4, r), piece % 4));
    return most > kMostByte;
  }
  // Row r of a matrix times `token(k)`, summed in binary64.
  template <typename T>
  static __device__ __forceinline__ float sum_again(const uint8_t *matrix, const void *scales, uint32_t n, uint32_t kblocks, uint32_t r, T token) {
    const uint8_t *row = matrix + static_cast<uint64_t>(r) * kblocks * kRowBytes;
    double sum = 0.0;
    for (uint32_t piece = 0; piece < kblocks * 4; ++piece) {  // of 32 values
      typedef float f2 __attribute__((ext_vector_type(2)));
      double of_piece = 0.0;
      for (uint32_t at = 0; at < 32; at += 2) {
        const f2 w = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(row[static_cast<uint64_t>(piece) * 16 + at / 2], 1.0f, 0);
        of_piece += static_cast<double>(w.x) * token(piece * 32 + at);
        of_piece += static_cast<double>(w.y) * token(piece * 32 + at + 1);
      }
      const uint32_t b = byte_of(scale(scales, n, piece / 4, r), piece % 4);
      sum += b < 255 ? ldexp(of_piece, static_cast<int>(b) - 127) : __builtin_nan("");
    }
    return static_cast<float>(sum);
  }
  static __device__ __forceinline__ f32x4 add(f32x4 acc, const bf16x8 *t, const bf16x8 *w, Scale) {
#pragma unroll
    for (int p = 0; p < 4; ++p) acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(t[p], w[p], acc, 0, 0, 0);
    return acc;
  }
};

struct F8 {
  static constexpr uint32_t kRowBytes = kBlock;
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
  static constexpr bool kSumsAgain = false;
  // A scale's power of two goes into the widened codes, its mantissa to the block's sum: codes are up to 448, so sums of codes
  // times x leave binary32's range where the weights' do not. (Powers from 2^-117 to 2^119 keep every code's product with them
  // a normal BF16 number, 2^-126 to 1.75 * 2^127; what a scale has beyond stays with the mantissa.)
  static __device__ __forceinline__ float power(Scale s) {
    constexpr uint32_t least = (127u - 117) << 23, most = (127u + 119) << 23;
    return __uint_as_float(min(max(__float_as_uint(s) & 0x7F800000u, least), most));
  }
  static __device__ __forceinline__ void widen(const Raw &r, Scale s, uint32_t, bf16x8 *f) {
    const float scale = power(s);
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const uint32_t x = r.w[p / 2][p % 2 * 2], y = r.w[p / 2][p % 2 * 2 + 1];
      const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x, scale, false), b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x, scale, true);
      const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(y, scale, false), d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(y, scale, true);
      f[p] = bf16x8{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
    }
  }
  static __device__ __forceinline__ f32x4 add(f32x4 acc, const bf16x8 *t, const bf16x8 *w, Scale s) {
    const float rest = s * __uint_as_float((254u << 23) - __float_as_uint(power(s)));  // over the power of two, exactly
    f32x4 c{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int p = 0; p < 4; ++p) c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(t[p], w[p], c, 0, 0, 0);
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] = __builtin_fmaf(c[e], rest, acc[e]);
    return acc;
  }
};

// The workspace: words[0] the number of experts in use; from words[kTable] on for
// each of those its number, the first place of its slots in the list, and how
// many they are; at words[kList] the list of slots, expert after expert, each
// expert's in order; then h, [2][slots][pitch], and y, [slots][pitch].
constexpr uint32_t kTable = 4, kList = kTable + 3 * kMaxGroups, kHidden = (kList + kMlpMaxSlots) * 4;
static_assert(kHidden % 16 == 0, "h is aligned");

constexpr uint32_t kWaves = 8, kMostRows = 64;  // of a wave's task

struct Args {
  const uint16_t *x;
  const void *ids;
  uint32_t wide;  // 64-bit ids
  const float *weights;
  const uint8_t *w;  // of this product: [experts][n][k]
  const void *scales;
  uint32_t *workspace;
  uint16_t *out;
  uint32_t tokens, topk, slots, experts;
  uint32_t cols, hidden, h_pitch, y_pitch;
  uint32_t n, k, kblocks;
  uint32_t strips;           // tasks that an expert's rows make
  uint32_t along, across;    // waves that share a row's blocks, and groups of them, each with rows of its own
  uint32_t segments, share;  // parts of k that the registers hold at a time; blocks of one that a wave takes
};

__device__ __forceinline__ uint16_t *h_of(const Args &p, uint32_t plane) {
  return reinterpret_cast<uint16_t *>(reinterpret_cast<uint8_t *>(p.workspace) + kHidden) + static_cast<uint64_t>(plane) * p.slots * p.h_pitch;
}
__device__ __forceinline__ float *y_of(const Args &p) { return reinterpret_cast<float *>(h_of(p, 2)); }

__device__ __forceinline__ uint32_t id_of(const Args &p, uint32_t slot) {
  // an id that is none counts as the expert past the last one
  const int64_t id = p.wide ? static_cast<const int64_t *>(p.ids)[slot] : static_cast<const int32_t *>(p.ids)[slot];
  return id < 0 || id >= p.experts ? p.experts : static_cast<uint32_t>(id);
}

// A row's first eight values, of which there are fewer.
__device__ __forceinline__ bf16x8 tokens_of_few(const uint16_t *row, uint32_t cols) {
  uint32_t e[8];
#pragma unroll
  for (uint32_t i = 0; i < 8; ++i) e[i] = i < cols ? row[i] : 0u;
  return __builtin_bit_cast(bf16x8, u32x4{e[0] | e[1] << 16, e[2] | e[3] << 16, e[4] | e[5] << 16, e[6] | e[7] << 16});
}

// Eight values without the first `drop`, and zeros behind them.
__device__ __forceinline__ bf16x8 without(bf16x8 v, uint32_t drop) {
  typedef uint64_t u64x2 __attribute__((ext_vector_type(2)));
  u64x2 w = __builtin_bit_cast(u64x2, v);
  const uint32_t bits = 16 * (drop % 4);
  const uint64_t carry = bits == 0 ? 0 : w.y << (64 - bits);
  const u64x2 near{w.x >> bits | carry, w.y >> bits};
  w = drop < 4 ? near : u64x2{near.y, 0};
  return __builtin_bit_cast(bf16x8, drop < 8 ? w : u64x2{0, 0});
}

// Far below zero, where 1 + e^-v is e^-v and from -88.7 on past the largest number, v e^v, of e^(v / 2) twice: e^v has no exponent
// left where the product has.
__device__ __forceinline__ float silu(float v) {
  const bool far = v < -80.0f;
  const float e = __expf(far ? 0.5f * v : -v);
  return far ? v * e * e : v / (1.0f + e);
}

// The experts in use, in order, and their slots.
struct Lists {
  uint32_t expert[kMaxGroups], start[kMaxGroups], count[kMaxGroups];
  uint32_t passes[kMaxGroups + 1];  // of `tokens` slots each, up to this expert's
  uint32_t in_use;
};

// passes from counts; one wave.
__device__ __forceinline__ void count_passes(Lists &l, uint32_t tokens) {
  const uint32_t lane = threadIdx.x % kWave;
  uint32_t n[4], scan = 0;
#pragma unroll
  for (uint32_t i = 0; i < 4; ++i) {
    n[i] = 4 * lane + i < l.in_use ? (l.count[4 * lane + i] + tokens - 1) / tokens : 0;
    scan += n[i];
  }
#pragma unroll
  for (uint32_t d = 1; d < kWave; d *= 2) {
    const uint32_t up = __shfl_up(scan, d);
    scan += lane >= d ? up : 0u;
  }
  uint32_t before = scan - n[0] - n[1] - n[2] - n[3];
  if (lane == 0) l.passes[0] = 0;
#pragma unroll
  for (uint32_t i = 0; i < 4; ++i) l.passes[4 * lane + i + 1] = before += n[i];
}

// The expert's slots number first .. first + most - 1, in order, to `to`; one wave.
__device__ __forceinline__ void slots_of(const uint16_t *ids, uint32_t slots, uint32_t expert, uint32_t first, uint32_t most, uint32_t *to) {
  const uint32_t lane = threadIdx.x % kWave;
  uint32_t count = 0;
  for (uint32_t s0 = 0; s0 < slots && count < first + most; s0 += kWave) {
    const bool mine = s0 + lane < slots && ids[s0 + lane] == expert;
    const uint64_t all = __ballot(mine);
    const uint32_t place = count + __popcll(all & ((uint64_t{1} << lane) - 1));
    if (mine && place >= first && place < first + most) to[place - first] = s0 + lane;
    count += __popcll(all);
  }
}

// U blocks along k a wave and segment at most, 16 MT tokens a pass, 16 NT rows a task. OUT: y from h, else h from x.
// WHOLE: k is a multiple of 8. SHORT: fewer than all waves share a row (else what depends on it is constant, which a token's layer
// takes 35.6 us with, not 36.6).
template <typename F, uint32_t U, uint32_t MT, uint32_t NT, bool OUT, bool GATED, bool WHOLE, bool SHORT>
__global__ __launch_bounds__(kWaves *kWave) void k_mlp(Args p) {
  constexpr uint32_t kPlanes = OUT ? 2 : 1, kTokens = 16 * MT;
  constexpr uint32_t kWide = GATED ? NT / 2 : NT, kGroups = MT * kWide;  // results of 16 x 16 of a task
  static_assert(16 * NT <= kMostRows, "what the pitches allow for");
  __shared__ f32x4 red[2][kWaves][NT][MT][kWave];
  __shared__ Lists lists;
  __shared__ uint16_t ids[OUT ? 1 : kMlpMaxSlots];
  __shared__ uint32_t of_pass[kWaves][kTokens];  // each wave's own copy
  __shared__ uint32_t again;                     // rows may have to be summed again
  const uint32_t lane = threadIdx.x % kWave, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const uint32_t i16 = lane % 16, q = lane / 16;
  const uint32_t along = SHORT ? p.along : kWaves, across = SHORT ? p.across : 1;
  const uint32_t wk = wave & (along - 1), wr = wave >> __builtin_ctz(along);

  if (OUT) {
    for (uint32_t i = threadIdx.x; i < kMaxGroups; i += kWaves * kWave) {
      lists.expert[i] = p.workspace[kTable + i];
      lists.start[i] = p.workspace[kTable + kMaxGroups + i];
      lists.count[i] = p.workspace[kTable + 2 * kMaxGroups + i];
    }
    if (threadIdx.x == 0) lists.in_use = p.workspace[0];
    __syncthreads();
  } else {
    // count every expert's slots, then number the experts that have some
    uint32_t *counts = reinterpret_cast<uint32_t *>(&red[0][0][0][0][0]);
    if (threadIdx.x < kMaxGroups) counts[threadIdx.x] = 0;
    lds_barrier();
    for (uint32_t s = threadIdx.x; s < p.slots; s += kWaves * kWave) {
      const uint32_t id = id_of(p, s);
      ids[s] = static_cast<uint16_t>(id);
      if (id < p.experts) atomicAdd(&counts[id], 1u);
    }
    lds_barrier();
    if (wave == 0) {
      uint32_t n[4], scan = 0;  // experts in use << 16 | slots
#pragma unroll
      for (uint32_t i = 0; i < 4; ++i) {
        n[i] = counts[4 * lane + i];
        scan += n[i] | (n[i] > 0 ? 1u << 16 : 0u);
      }
      const uint32_t own = scan;
#pragma unroll
      for (uint32_t d = 1; d < kWave; d *= 2) {
        const uint32_t up = __shfl_up(scan, d);
        scan += lane >= d ? up : 0u;
      }
      uint32_t rank = (scan - own) >> 16, start = (scan - own) & 0xFFFF;
#pragma unroll
      for (uint32_t i = 0; i < 4; ++i) {
        if (n[i] == 0) continue;
        lists.expert[rank] = 4 * lane + i;
        lists.start[rank] = start;
        lists.count[rank] = n[i];
        ++rank, start += n[i];
      }
      if (lane == kWave - 1) lists.in_use = scan >> 16;
    }
    lds_barrier();
    // the second kernel's copy: a workgroup writes down the lists of every so-manyth expert
    const uint32_t in_use = __builtin_amdgcn_readfirstlane(lists.in_use);
    if (blockIdx.x == 0 && threadIdx.x == 0) p.workspace[0] = in_use;
    if (wave == kWaves - 1) {
      for (uint32_t r = blockIdx.x; r < in_use; r += gridDim.x) {
        const uint32_t expert = __builtin_amdgcn_readfirstlane(lists.expert[r]), start = __builtin_amdgcn_readfirstlane(lists.start[r]);
        const uint32_t count = __builtin_amdgcn_readfirstlane(lists.count[r]);
        if (lane == 0) {
          p.workspace[kTable + r] = expert;
          p.workspace[kTable + kMaxGroups + r] = start;
          p.workspace[kTable + 2 * kMaxGroups + r] = count;
        }
        slots_of(ids, p.slots, expert, 0, count, p.workspace + kList + start);
      }
    }
  }
  if (wave == 0) count_passes(lists, kTokens);
  if (F::kSumsAgain && threadIdx.x == 0) again = 0;
  lds_barrier();

  // this workgroup's tasks: pass after pass, strip after strip
  const uint64_t tasks = static_cast<uint64_t>(__builtin_amdgcn_readfirstlane(lists.passes[kMaxGroups])) * p.strips;
  const uint64_t first_task = tasks * blockIdx.x / gridDim.x, end_task = tasks * (blockIdx.x + 1) / gridDim.x;
  if (first_task >= end_task) return;

  struct Task {
    uint32_t pass, strip, segment;
    uint32_t rank, expert;
  };
  auto settle = [&](Task &t) {  // the pass's expert
    while (t.pass >= __builtin_amdgcn_readfirstlane(lists.passes[t.rank + 1])) ++t.rank;
    t.expert = __builtin_amdgcn_readfirstlane(lists.expert[t.rank]);
  };
  const uint64_t pitch = static_cast<uint64_t>(p.kblocks) * F::kRowBytes, scale_bytes = F::scale_bytes(p.n, p.kblocks);
  typename F::Raw raw[U][NT];
  typename F::Scale scale[U][NT];
  struct From {
    const uint8_t *row[NT];
    const uint8_t *scales;
    uint32_t at[NT];  // rows of the matrix; those past the end repeat the last one, and their results are not used
  };
  auto block_of = [&](uint32_t segment, uint32_t u) { return (segment * along + wk) * p.share + u; };
  auto from_of = [&](const Task &t) {
    From f;
    const uint8_t *matrix = p.w + static_cast<uint64_t>(t.expert) * p.n * pitch;
    f.scales = static_cast<const uint8_t *>(p.scales) + t.expert * scale_bytes;
#pragma unroll
    for (uint32_t i = 0; i < NT; ++i) {
      f.at[i] = min(((t.strip * across + wr) * kWide + i % kWide) * 16 + i16, (OUT ? p.n : p.hidden) - 1) + i / kWide * p.hidden;
      f.row[i] = matrix + f.at[i] * pitch;
    }
    return f;
  };
  auto load = [&](const From &f, const Task &t, uint32_t u, uint32_t i) {
    const uint32_t kb = min(block_of(t.segment, min(u, p.share - 1)), p.kblocks - 1);  // past the end: loaded again, not used
    raw[u][i] = F::load(f.row[i] + static_cast<uint64_t>(kb) * F::kRowBytes, q);
    scale[u][i] = F::scale(f.scales, p.n, kb, f.at[i]);
  };
  bf16x8 tok[U][MT][kPlanes][4];
  uint32_t count = 0;  // the pass's tokens
  auto list_tokens = [&](const Task &t) {
    const uint32_t first = (t.pass - __builtin_amdgcn_readfirstlane(lists.passes[t.rank])) * kTokens;
    count = min(kTokens, __builtin_amdgcn_readfirstlane(lists.count[t.rank]) - first);
    if (OUT) {
      if (lane < count) of_pass[wave][lane] = p.workspace[kList + lists.start[t.rank] + first + lane];
    } else {
      slots_of(ids, p.slots, t.expert, first, kTokens, of_pass[wave]);
    }
    __builtin_amdgcn_wave_barrier();
  };
  auto load_tokens = [&](const Task &t) {
    list_tokens(t);
    const uint16_t *row[MT];
#pragma unroll
    for (uint32_t m = 0; m < MT; ++m) {
      const uint32_t slot = of_pass[wave][min(16 * m + i16, count - 1)];
      row[m] = OUT ? h_of(p, 0) + static_cast<uint64_t>(slot) * p.h_pitch : p.x + static_cast<uint64_t>(slot / p.topk) * p.cols;
    }
    const uint64_t plane = OUT ? static_cast<uint64_t>(p.slots) * p.h_pitch : 0;
    if constexpr (WHOLE) {  // pieces of eight are whole, or past the end
#pragma unroll
      for (uint32_t u = 0; u < U; ++u) {
        const uint32_t kb = min(block_of(t.segment, min(u, p.share - 1)), p.kblocks - 1);
#pragma unroll
        for (uint32_t m = 0; m < MT; ++m)
#pragma unroll
          for (uint32_t l = 0; l < kPlanes; ++l)
#pragma unroll
            for (uint32_t e = 0; e < 4; ++e) {
              const uint32_t at = kb * kBlock + F::at(q, e);
              const u32x4 w = *reinterpret_cast<const u32x4 *>(row[m] + l * plane + (OUT ? at : min(at, p.cols - 8)));
              tok[u][m][l][e] = __builtin_bit_cast(bf16x8, OUT || at < p.cols ? w : u32x4{0, 0, 0, 0});
            }
      }
    } else if (p.cols < 8) {
#pragma unroll
      for (uint32_t u = 0; u < U; ++u)
#pragma unroll
        for (uint32_t m = 0; m < MT; ++m)
#pragma unroll
          for (uint32_t e = 0; e < 4; ++e)
            tok[u][m][0][e] = e == 0 && q == 0 ? tokens_of_few(row[m], p.cols) : __builtin_bit_cast(bf16x8, u32x4{0, 0, 0, 0});
    } else {
      // Rows start anywhere, which the loads may; a piece that ends past the row is the row's last eight, some of them dropped.
      // (Value by value, 64 tokens and 2 x 512 x 4100 in MXFP4 took 160 us, not 92.)
#pragma unroll
      for (uint32_t u = 0; u < U; ++u) {
        const uint32_t kb = min(block_of(t.segment, min(u, p.share - 1)), p.kblocks - 1);
#pragma unroll
        for (uint32_t m = 0; m < MT; ++m)
#pragma unroll
          for (uint32_t e = 0; e < 4; ++e) {
            const uint32_t at = kb * kBlock + F::at(q, e), from = min(at, p.cols - 8);
            const u32x4 w = *reinterpret_cast<const u32x4_any *>(row[m] + from);
            tok[u][m][0][e] = without(__builtin_bit_cast(bf16x8, w), at - from);
          }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
  };

  // Column c of a slot's row, from its row's sum and, gated, the second half's (asked for when the first is done with: both at a time
  // are more than the registers hold).
  auto put = [&](uint32_t slot, uint32_t c, float v, auto up) {
    if (OUT) {
      if (c < p.y_pitch) y_of(p)[static_cast<uint64_t>(slot) * p.y_pitch + c] = v;
      return;
    }
    // units past the last one, up to the block's end, are zeros
    const float h = c < p.hidden ? (GATED ? silu(v) * up() : silu(v)) : 0.0f;
    if (c < p.h_pitch) {
      const uint64_t at = static_cast<uint64_t>(slot) * p.h_pitch + c;
      uint32_t hi = bf16_pair(h, 0.0f) & 0xFFFF;
      if ((hi & 0x7FFF) == 0x7F80 && fabsf(h) < __builtin_inff()) --hi;  // (past BF16's largest number by less than a step: that number)
      // (where h is no number, or infinite, so that the sum shall be, the rest is nothing)
      const float rest = h - __uint_as_float(hi << 16);
      h_of(p, 0)[at] = static_cast<uint16_t>(hi);
      h_of(p, 1)[at] = static_cast<uint16_t>(bf16_pair(rest == rest ? rest : 0.0f, 0.0f));
    }
  };

  // A finished task's sums wait in LDS until late in the next one, when every wave's have long been there: the
  // waves do not wait for each other, and the next weights are on their way meanwhile.
  uint32_t buffer = 0, waiting = 0;  // strip + 1 of the task that waits
  auto finish = [&] {
    if (waiting == 0) return;
    lds_barrier();
    const uint32_t strip = waiting - 1;
    waiting = 0;
    for (uint32_t it = wave; it < 4 * kGroups * across; it += kWaves) {
      const uint32_t rows = it / (4 * kGroups), group = it / 4 % kGroups, e = it % 4, m = group / kWide, i = group % kWide;
      auto sum = [&](uint32_t i) {
        const f32x4(*from)[NT][MT][kWave] = &red[buffer ^ 1][rows * along];
        float v = from[0][i][m][lane][e];
#pragma unroll
        for (uint32_t k = 1; k < kWaves; ++k) {
          if (k == along) break;
          v += from[k][i][m][lane][e];
        }
        return v;
      };
      const uint32_t place = 16 * m + 4 * q + e, c = ((strip * across + rows) * kWide + i) * 16 + i16;
      const float v = sum(i);
      if (place < count) put(of_pass[wave][place], c, v, [&] { return sum(kWide + i); });
    }
  };

  Task now{static_cast<uint32_t>(first_task / p.strips), static_cast<uint32_t>(first_task % p.strips), 0, 0, 0};
  settle(now);
  {
    const From f = from_of(now);
#pragma unroll
    for (uint32_t i = 0; i < NT; ++i)
#pragma unroll
      for (uint32_t u = 0; u < U; ++u) load(f, now, u, i);
  }
  load_tokens(now);
  f32x4 acc[MT][NT];
  uint32_t most = 0;  // scale byte that this lane has seen
  for (uint64_t task = first_task; task < end_task;) {
    if (now.segment == 0) {
#pragma unroll
      for (uint32_t m = 0; m < MT; ++m)
#pragma unroll
        for (uint32_t i = 0; i < NT; ++i) acc[m][i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    Task next = now;
    const bool last_segment = ++next.segment == p.segments;
    if (last_segment) {
      next.segment = 0;
      if (++next.strip == p.strips) next.strip = 0, ++next.pass;
    }
    const bool more = !last_segment || task + 1 < end_task;
    if (more) settle(next);
    From f = from_of(more ? next : now);
    if (!more) {  // nothing is left to load: a line that all of the wave reads
#pragma unroll
      for (uint32_t i = 0; i < NT; ++i) f.row[i] = p.w;
    }
#pragma unroll
    for (uint32_t i = 0; i < NT; ++i) {
      if (i == NT - 1) finish();
#pragma unroll
      for (uint32_t u = 0; u < U; ++u) {
        const bool used = u < p.share && block_of(now.segment, u) < p.kblocks;
        bf16x8 w[4];
        const typename F::Scale s = scale[u][i];
        F::widen(raw[u][i], s, q, w);
        if constexpr (F::kSumsAgain) F::watch(most, s, q);
        // (widened by now: else the old registers would live past the loads, and be copied, all loads waited for, each task)
        asm volatile("" : "+v"(w[0]), "+v"(w[1]), "+v"(w[2]), "+v"(w[3])::"memory");
        load(f, next, u, i);
        if (!used) continue;
#pragma unroll
        for (uint32_t m = 0; m < MT; ++m)
#pragma unroll
          for (uint32_t l = 0; l < kPlanes; ++l) acc[m][i] = F::add(acc[m][i], tok[u][m][l], w, s);
      }
    }
    if (last_segment) {
#pragma unroll
      for (uint32_t m = 0; m < MT; ++m)
#pragma unroll
        for (uint32_t i = 0; i < NT; ++i) red[buffer][wave][i][m][lane] = acc[m][i];
      buffer ^= 1;
      waiting = now.strip + 1;
      ++task;
    }
    const bool other_tokens = more && (p.segments > 1 || next.pass != now.pass);
    if (!more || (other_tokens && next.pass != now.pass)) finish();  // of this pass's tokens
    if (other_tokens) load_tokens(next);
    now = next;
  }

  if constexpr (F::kSumsAgain) {
    if (__any(most > F::kMostByte)) again = 1;
    __syncthreads();  // (and all results are stored)
    if (__builtin_amdgcn_readfirstlane(again) == 0) return;
    const uint32_t wide = across * kWide * 16;  // columns of a task
    Task t{0, 0, 0, 0, 0};
    for (uint64_t task = first_task; task < end_task; ++task) {
      t.pass = static_cast<uint32_t>(task / p.strips), t.strip = static_cast<uint32_t>(task % p.strips);
      settle(t);
      list_tokens(t);
      const uint8_t *matrix = p.w + static_cast<uint64_t>(t.expert) * p.n * pitch, *scales = static_cast<const uint8_t *>(p.scales) + t.expert * scale_bytes;
      for (uint32_t it = threadIdx.x; it < wide * count; it += kWaves * kWave) {
        const uint32_t slot = of_pass[wave][it / wide], c = t.strip * wide + it % wide;
        if (c >= (OUT ? p.n : p.hidden)) continue;
        auto token = [&](uint32_t k) {
          if (OUT) return bf16_lo(h_of(p, 0)[static_cast<uint64_t>(slot) * p.h_pitch + k]) + bf16_lo(h_of(p, 1)[static_cast<uint64_t>(slot) * p.h_pitch + k]);
          return k < p.cols ? bf16_lo(p.x[static_cast<uint64_t>(slot / p.topk) * p.cols + k]) : 0.0f;
        };
        if (!F::row_lacks(scales, p.n, p.kblocks, c) && !(GATED && F::row_lacks(scales, p.n, p.kblocks, c + p.hidden))) continue;
        const float v = F::sum_again(matrix, scales, p.n, p.kblocks, c, token);
        put(slot, c, v, [&] { return F::sum_again(matrix, scales, p.n, p.kblocks, c + p.hidden, token); });
      }
    }
  }
}

// ---------------------------------------------------------------------------
// out: four columns of a token to a thread, its slots in the order of the choices, one after the other (a choice that is left out
// is a branch, so each one's loads wait for those before).
// ---------------------------------------------------------------------------
constexpr uint32_t kCombineThreads = 256;
__global__ __launch_bounds__(kCombineThreads) void k_mlp_combine(Args p, uint32_t per_row) {
  const uint32_t t = blockIdx.x / per_row, c = (blockIdx.x % per_row * kCombineThreads + threadIdx.x) * 4;
  if (c >= p.cols) return;
  const float *y = y_of(p);
  f32x4 v{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
  for (uint32_t j = 0; j < p.topk; ++j) {
    const uint32_t slot = t * p.topk + j;
    if (id_of(p, slot) == p.experts) continue;
    v += p.weights[slot] * *reinterpret_cast<const f32x4 *>(y + static_cast<uint64_t>(slot) * p.y_pitch + c);
  }
  store4<false>(p.out, static_cast<uint64_t>(t) * p.cols, c, p.cols, v);
}

uint32_t h_pitch(uint64_t hidden) { return static_cast<uint32_t>((hidden + kBlock - 1) / kBlock * kBlock); }
uint32_t y_pitch(uint64_t cols) { return static_cast<uint32_t>((cols + kMostRows - 1) / kMostRows * kMostRows); }

constexpr uint32_t kWorkgroups = 256;  // one a CU

template <typename F, uint32_t U, uint32_t MT, uint32_t NT, bool OUT, bool WHOLE = true>
hipError_t launch_product(Args a, bool gated, hipStream_t s) {
  a.kblocks = (a.k + kBlock - 1) / kBlock;
  // rows of h up to the end of its last block, so that what the second kernel reads is written
  const uint32_t wide = gated ? 8 * NT : 16 * NT, results = OUT ? a.y_pitch : a.h_pitch;
  // Rows shorter than what eight waves hold are shared by fewer, which take more rows at a time, while there is a task for
  // every CU. A layer of 64 tokens, 64 experts of 2 x 512 x 4096 in MXFP4 78 -> 62 us, 2 x 512 x 1024 43 -> 35; of 128 tokens
  // and 2 x 2944 x 128 in FP8 117 -> 49.
  constexpr bool kMayBeShort = U == 2;  // (the other kernels are for rows that are not)
  for (a.along = kMayBeShort ? 1 : kWaves;; a.along *= 2) {
    a.across = kWaves / a.along;
    a.strips = (results + wide * a.across - 1) / (wide * a.across);
    if (a.along == kWaves || (a.kblocks <= a.along * U && static_cast<uint64_t>(min(a.experts, a.slots)) * a.strips >= kWorkgroups)) break;
  }
  a.segments = (a.kblocks + a.along * U - 1) / (a.along * U);
  a.share = (a.kblocks + a.along * a.segments - 1) / (a.along * a.segments);
  const uint64_t passes = min(a.experts, a.slots) + a.slots / (16 * MT);
  const dim3 grid(static_cast<uint32_t>(min(static_cast<uint64_t>(kWorkgroups), passes * a.strips)));
  if (kMayBeShort && a.along < kWaves) {
    if (gated) hipLaunchKernelGGL((k_mlp<F, U, MT, NT, OUT, !OUT, WHOLE, kMayBeShort>), grid, dim3(kWaves * kWave), 0, s, a);
    else hipLaunchKernelGGL((k_mlp<F, U, MT, NT, OUT, false, WHOLE, kMayBeShort>), grid, dim3(kWaves * kWave), 0, s, a);
  } else if (gated) {
    hipLaunchKernelGGL((k_mlp<F, U, MT, NT, OUT, !OUT, WHOLE, false>), grid, dim3(kWaves * kWave), 0, s, a);
  } else {
    hipLaunchKernelGGL((k_mlp<F, U, MT, NT, OUT, false, WHOLE, false>), grid, dim3(kWaves * kWave), 0, s, a);
  }
  return hipGetLastError();
}

// What the registers hold of a wave's share of k: blocks U times tokens 16 MT (times two numbers for h), and weights
// U times rows 16 NT. Which MT, by the slots an expert on average over all experts (how they spread is not known here): one pass of 32
// slots against two of 16, where most experts have more than 16. Times in us with MT 1 / 2, weights from HBM:
//   slots an expert                      8          12         16         20         24         32         48         64         128
//   32 experts of 2 x 1024 x 1024, FP8   39 / 43    51 / 44    54 / 46    59 / 48    64 / 63    71 / 70
//     MXFP4                              33 / 36    42 / 38    45 / 39    49 / 42    51 / 56    58 / 64
//   8 experts of 2 x 768 x 2048, FP8     28 / 28    31 / 30    39 / 31    38 / 32    38 / 35    46 / 47    55 / 44    63 / 57    77 / 57
//     MXFP4                              23 / 25    26 / 26    32 / 28    32 / 29    31 / 31    39 / 42    45 / 39    50 / 51
//   64 experts of 2 x 1024 x 2048, FP8              104 / 104  117 / 106;  MXFP4 76 / 77  87 / 80
// so from 12 on; where some experts' slots pass 32 and take two passes of 32 (24 to 32 on average) MXFP4 loses up to a tenth by it.
// Longer rows than the registers hold go in segments, and their tokens are loaded again for each: FP8 takes 16 tokens for those.
// (MXFP4, 32 experts of 2 x 1024, 32 tokens for 4 each: 4096 columns 60 us, 4104 80, 8192 113; the weights at a copy's rate 42, 41, 84.)
hipError_t launch_hidden(const Args &a, bool fp8, bool gated, hipStream_t s) {
  const bool two = a.slots > 12 * a.experts;
  const uint32_t share = (a.k + kBlock * kWaves - 1) / (kBlock * kWaves);
  if (a.k % 8 != 0) {  // (with U 4 and 5 no faster: 2 x 512 x 4100 92 / 91 us, one token's 29.4 / 30.9)
    if (fp8) return two ? launch_product<F8, 2, 2, 4, false, false>(a, gated, s) : launch_product<F8, 2, 1, 4, false, false>(a, gated, s);
    return two ? launch_product<Mx, 2, 2, 4, false, false>(a, gated, s) : launch_product<Mx, 2, 1, 4, false, false>(a, gated, s);
  }
  if (fp8) {
    if (share > 2) return launch_product<F8, 5, 1, 2, false>(a, gated, s);
    return two ? launch_product<F8, 2, 2, 4, false>(a, gated, s) : launch_product<F8, 2, 1, 4, false>(a, gated, s);
  }
  if (two) return share <= 2 ? launch_product<Mx, 2, 2, 4, false>(a, gated, s) : launch_product<Mx, 4, 2, 2, false>(a, gated, s);
  return share <= 2 ? launch_product<Mx, 2, 1, 4, false>(a, gated, s) : launch_product<Mx, 4, 1, 4, false>(a, gated, s);
}
hipError_t launch_out(const Args &a, bool fp8, hipStream_t s) {
  const bool two = a.slots > 12 * a.experts;
  const uint32_t share = (a.k + kBlock * kWaves - 1) / (kBlock * kWaves);
  if (fp8) return two && share <= 2 ? launch_product<F8, 2, 2, 2, true>(a, false, s) : launch_product<F8, 2, 1, 4, true>(a, false, s);
  if (share > 2) return launch_product<Mx, 4, 1, 2, true>(a, false, s);
  return two ? launch_product<Mx, 2, 2, 2, true>(a, false, s) : launch_product<Mx, 2, 1, 4, true>(a, false, s);
}

}  // namespace

uint64_t expert_mlp_workspace_bytes(uint64_t slots, uint64_t cols, uint64_t hidden) {
  return kHidden + slots * (4 * static_cast<uint64_t>(h_pitch(hidden)) + 4 * static_cast<uint64_t>(y_pitch(cols)));
}

hipError_t launch_expert_mlp(const ExpertMlp &p, hipStream_t s) {
  Args a{};
  a.x = static_cast<const uint16_t *>(p.x);
  a.ids = p.ids;
  a.wide = p.wide;
  a.weights = p.weights;
  a.workspace = p.workspace;
  a.out = static_cast<uint16_t *>(p.out);
  a.tokens = p.tokens;
  a.topk = p.topk;
  a.slots = p.tokens * p.topk;
  a.experts = p.experts;
  a.cols = p.cols;
  a.hidden = p.hidden;
  a.h_pitch = h_pitch(p.hidden);
  a.y_pitch = y_pitch(p.cols);
  a.w = p.w1;
  a.scales = p.s1;
  a.n = p.hidden * (p.gated ? 2 : 1);
  a.k = p.cols;
  hipError_t e = launch_hidden(a, p.fp8, p.gated, s);
  if (e != hipSuccess) return e;
  a.w = p.w2;
  a.scales = p.s2;
  a.n = p.cols;
  a.k = p.hidden;
  if ((e = launch_out(a, p.fp8, s)) != hipSuccess) return e;
  const uint32_t per_row = (p.cols + 4 * kCombineThreads - 1) / (4 * kCombineThreads);
  hipLaunchKernelGGL(k_mlp_combine, dim3(p.tokens * per_row), dim3(kCombineThreads), 0, s, a, per_row);
  return hipGetLastError();
}

}  // namespace nvfp4
