// Tokens sorted by expert and back, and the gradients of both.
//
// A router gives every token topk experts. Choice j of token t is slot
// t * topk + j. The sort puts the slots of one expert next to each other
// (stable: by slot), each expert's rows starting at a multiple of `align`,
// so that the sorted rows are the groups of a grouped quantize or product.
// Rows between an expert's last token and the next expert's first one, and
// past the last expert, are padding.
//
//   gather           y[r] = x[row_slots[r] / topk], 0 in padding
//   combine          out[t] = sum_j w[t][j] * y[slot_rows[t][j]]
//   combine's grads  dy[r] = w[s] * dout[s / topk], 0 in padding;
//                    dw[s] = <dout[s / topk], y[slot_rows[s]]>
//   gather's grad    dx[t] = sum_j dy[slot_rows[t][j]]: combine without w
//
// Dropped slots (an id outside 0 .. experts - 1) have slot_rows -1 and are
// left out of every sum; their dw is 0. Sums are held in binary32, in the
// order j = 0, 1, ..; nothing uses floating-point atomics, so a call gives
// the same bits every time.
#include <algorithm>

#include "codec.h"
#include "launch.h"

namespace nvfp4 {
namespace {

constexpr uint32_t kWave = 64;

// ---------------------------------------------------------------------------
// Sort: a counting sort over at most kMaxKeys keys. A workgroup of 16
// waves takes a chunk of slots; inside it each wave takes consecutive slots,
// 64 at a time, and ranks them by matching keys across its lanes (eight
// ballots, one for each bit of the key), so ranks follow the slots' order
// and no atomic decides it. Up to kSortTile slots one launch does all; more
// take a launch that counts each chunk's keys first. The work is a few bytes
// a slot: what bounds it is the latency of its steps, not bandwidth.
// ---------------------------------------------------------------------------
constexpr uint32_t kSortThreads = 1024;
constexpr uint32_t kSortWaves = kSortThreads / kWave;
constexpr uint32_t kSortRounds = 4;                              // 64-slot rounds of a wave in one tile
constexpr uint32_t kSortTile = kSortThreads * kSortRounds;       // slots of one tile
constexpr uint32_t kSortChunks = 256;                            // most chunks (workgroups) of a sort
constexpr uint32_t kMaxKeys = kMaxGroups;

struct SortArgs {
  const void *ids;
  uint32_t wide;  // ids are 64-bit
  uint32_t slots, experts, align_log2;
  uint32_t chunk, chunks;  // slots of a chunk, chunks
  uint32_t rounds;         // rounds of a wave in a tile
  uint32_t rows;
  int32_t *slot_rows, *row_slots, *offsets, *counts;
  uint32_t *hist;  // [chunks][experts]; NULL with one chunk
};

// The slot's expert, or kMaxKeys for one that is dropped.
__device__ __forceinline__ uint32_t load_key(const SortArgs &a, uint32_t slot) {
  if (a.wide) {
    const int64_t id = static_cast<const int64_t *>(a.ids)[slot];
    return id >= 0 && id < static_cast<int64_t>(a.experts) ? static_cast<uint32_t>(id) : kMaxKeys;
  }
  const uint32_t id = static_cast<const uint32_t *>(a.ids)[slot];  // negative ids are large here
  return id < a.experts ? id : kMaxKeys;
}

__global__ __launch_bounds__(kSortThreads) void k_expert_count(SortArgs a) {
  __shared__ uint32_t hist[kMaxKeys + 1];
  for (uint32_t i = threadIdx.x; i <= kMaxKeys; i += kSortThreads) hist[i] = 0;
  __syncthreads();
  const uint64_t first = static_cast<uint64_t>(blockIdx.x) * a.chunk;
  const uint64_t last = min(first + a.chunk, static_cast<uint64_t>(a.slots));
  for (uint64_t i = first + threadIdx.x; i < last; i += kSortThreads) atomicAdd(&hist[load_key(a, static_cast<uint32_t>(i))], 1u);
  __syncthreads();
  for (uint32_t e = threadIdx.x; e < a.experts; e += kSortThreads) a.hist[blockIdx.x * a.experts + e] = hist[e];
}

__global__ __launch_bounds__(kSortThreads) void k_expert_place(SortArgs a) {
  __shared__ uint32_t cnt[kSortWaves][kMaxKeys];  // a wave's slots of each key; then its first rank
  __shared__ uint32_t total[kMaxKeys], next[kMaxKeys], start[kMaxKeys + 1], parts[kSortThreads / kMaxKeys][2][kMaxKeys];
  const uint32_t t = threadIdx.x, lane = t % kWave, wave = t / kWave;
  const uint64_t first = static_cast<uint64_t>(blockIdx.x) * a.chunk;
  const uint64_t last = min(first + a.chunk, static_cast<uint64_t>(a.slots));
  const uint64_t below = (uint64_t{1} << lane) - 1;

  for (uint64_t tile = first; tile < last || tile == first; tile += kSortWaves * kWave * a.rounds) {
    for (uint32_t i = t; i < kSortWaves * kMaxKeys; i += kSortThreads) cnt[i / kMaxKeys][i % kMaxKeys] = 0;
    __syncthreads();
    uint32_t key[kSortRounds], rank[kSortRounds];
#pragma unroll
    for (uint32_t r = 0; r < kSortRounds; ++r) {
      const uint64_t slot = tile + (wave * a.rounds + r) * kWave + lane;
      key[r] = r < a.rounds && slot < last ? load_key(a, static_cast<uint32_t>(slot)) : kMaxKeys;
    }
#pragma unroll
    for (uint32_t r = 0; r < kSortRounds; ++r) {
      if (r >= a.rounds) break;
      const bool valid = key[r] < kMaxKeys;
      uint64_t same = __ballot(valid);
#pragma unroll
      for (uint32_t bit = 0; bit < 8; ++bit) {
        const bool one = (key[r] >> bit) & 1u;
        const uint64_t ones = __ballot(one);
        same &= one ? ones : ~ones;
      }
      rank[r] = 0;
      if (valid) {
        // LDS operations of one wave are done in order: every lane reads the
        // count before the first lane of its key adds to it
        const uint32_t before = cnt[wave][key[r]];
        rank[r] = before + __popcll(same & below);
        if ((same & below) == 0) cnt[wave][key[r]] = before + __popcll(same);
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // the next round reads what other lanes wrote
    }
    __syncthreads();
    if (tile == first) {
      // totals, this chunk's first rank of each key, and the experts' first rows
      if (a.hist == nullptr) {
        if (t < kMaxKeys) {
          uint32_t all = 0;
#pragma unroll
          for (uint32_t w = 0; w < kSortWaves; ++w) all += cnt[w][t];
          total[t] = all;
          next[t] = 0;
        }
      } else {  // four threads a key, each a quarter of the chunks
        const uint32_t e = t % kMaxKeys, part = t / kMaxKeys;
        uint32_t mine = 0, all = 0;
        if (e < a.experts) {
#pragma unroll 8
          for (uint32_t c = part; c < a.chunks; c += kSortThreads / kMaxKeys) {
            const uint32_t h = a.hist[c * a.experts + e];
            all += h;
            mine += c < blockIdx.x ? h : 0u;
          }
        }
        parts[part][0][e] = all;
        parts[part][1][e] = mine;
        __syncthreads();
        if (t < kMaxKeys) {
          total[t] = parts[0][0][t] + parts[1][0][t] + parts[2][0][t] + parts[3][0][t];
          next[t] = parts[0][1][t] + parts[1][1][t] + parts[2][1][t] + parts[3][1][t];
        }
      }
      __syncthreads();
      if (wave == 0) {  // exclusive sum of the padded totals, four keys a lane
        uint32_t v[4], sum = 0;
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i) {
          v[i] = sum;
          sum += ((total[4 * lane + i] + (1u << a.align_log2) - 1) >> a.align_log2) << a.align_log2;
        }
        uint32_t scan = sum;
#pragma unroll
        for (uint32_t d = 1; d < kWave; d *= 2) {
          const uint32_t up = __shfl_up(scan, d);
          scan += lane >= d ? up : 0u;
        }
#pragma unroll
        for (uint32_t i = 0; i < 4; ++i) start[4 * lane + i] = scan - sum + v[i];
        if (lane == kWave - 1) start[kMaxKeys] = scan;
      }
      __syncthreads();
    }
    if (t < kMaxKeys) {  // each wave's first rank of each key
      uint32_t n = next[t];
#pragma unroll
      for (uint32_t w = 0; w < kSortWaves; ++w) {
        const uint32_t c = cnt[w][t];
        cnt[w][t] = n;
        n += c;
      }
      next[t] = n;
    }
    __syncthreads();
#pragma unroll
    for (uint32_t r = 0; r < kSortRounds; ++r) {
      const uint64_t slot = tile + (wave * a.rounds + r) * kWave + lane;
      if (r >= a.rounds || slot >= last) continue;
      int32_t row = -1;
      if (key[r] < kMaxKeys) {
        const uint32_t at = start[key[r]] + cnt[wave][key[r]] + rank[r];
        if (at < a.rows) {  // always, if nothing writes the ids meanwhile
          row = static_cast<int32_t>(at);
          a.row_slots[at] = static_cast<int32_t>(slot);
        }
      }
      a.slot_rows[slot] = row;
    }
    __syncthreads();
  }

  // padding: each expert's by one wave, what follows the last expert by all
  for (uint32_t e = blockIdx.x * kSortWaves + wave; e < a.experts; e += a.chunks * kSortWaves) {
    const uint32_t end = min(start[e + 1], a.rows);
    for (uint32_t r = start[e] + total[e] + lane; r < end; r += kWave) a.row_slots[r] = -1;
  }
  for (uint64_t r = static_cast<uint64_t>(start[a.experts]) + blockIdx.x * kSortThreads + t; r < a.rows; r += a.chunks * kSortThreads)
    a.row_slots[r] = -1;
  if (blockIdx.x == 0) {
    for (uint32_t e = t; e <= a.experts; e += kSortThreads) a.offsets[e] = static_cast<int32_t>(start[e]);
    for (uint32_t e = t; e < a.experts; e += kSortThreads) a.counts[e] = static_cast<int32_t>(total[e]);
  }
}

// ---------------------------------------------------------------------------
// Rows of BF16 or FP32 in pieces of 16 bytes. With an odd number of columns
// rows start at any element, so the pieces are only element-aligned, which
// global loads and stores take (at some cost); the rest of a row shorter
// than a piece goes element by element.
// ---------------------------------------------------------------------------
typedef uint32_t piece_t __attribute__((ext_vector_type(4), aligned(2)));

template <int DT>
struct Elem;
template <>
struct Elem<kBF16> {
  typedef uint16_t type;
  static constexpr uint32_t per = 8;
  static __device__ __forceinline__ float load(const type *p) { return __uint_as_float(static_cast<uint32_t>(*p) << 16); }
  static __device__ __forceinline__ void store(type *p, float v) { *p = static_cast<type>(bf16_pair(v, 0.0f)); }
  static __device__ __forceinline__ void unpack(piece_t v, float *f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = bf16_lo(v[i]);
      f[2 * i + 1] = bf16_hi(v[i]);
    }
  }
  static __device__ __forceinline__ piece_t pack(const float *f) {
    piece_t v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = bf16_pair(f[2 * i], f[2 * i + 1]);
    return v;
  }
};
template <>
struct Elem<kFP32> {
  typedef float type;
  static constexpr uint32_t per = 4;
  static __device__ __forceinline__ float load(const type *p) { return *p; }
  static __device__ __forceinline__ void store(type *p, float v) { *p = v; }
  static __device__ __forceinline__ void unpack(piece_t v, float *f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(v[i]);
  }
  static __device__ __forceinline__ piece_t pack(const float *f) {
    piece_t v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = __float_as_uint(f[i]);
    return v;
  }
};

constexpr uint32_t kRowThreads = 256;
constexpr uint32_t kRowWaves = kRowThreads / kWave;

__device__ __forceinline__ uint32_t wave_index() { return __builtin_amdgcn_readfirstlane(threadIdx.x / kWave); }

template <int DT>
__device__ __forceinline__ void zero_row(typename Elem<DT>::type *dst, uint32_t cols, uint32_t lane) {
  constexpr uint32_t per = Elem<DT>::per;
  for (uint32_t c = lane * per; c + per <= cols; c += kWave * per) *reinterpret_cast<piece_t *>(dst + c) = piece_t{0, 0, 0, 0};
  for (uint32_t c = cols / per * per + lane; c < cols; c += kWave) dst[c] = 0;
}

// A row's pieces past the caches: rows that are written or read once.
__device__ __forceinline__ void put(void *p, piece_t v) { __builtin_nontemporal_store(v, static_cast<piece_t *>(p)); }
__device__ __forceinline__ piece_t take(const void *p) { return __builtin_nontemporal_load(static_cast<const piece_t *>(p)); }

// Rows without a slot are cleared by waves of their own, kPadRows of them each.
constexpr uint32_t kPadRows = 2;
template <int DT>
__device__ __forceinline__ void clear_padding(typename Elem<DT>::type *y, const int32_t *row_slots, uint64_t r0, uint32_t slots,
                                              uint32_t cols, uint32_t rows, uint32_t lane) {
  for (uint64_t r = r0; r < r0 + kPadRows && r < rows; ++r)
    if (static_cast<uint32_t>(row_slots[r]) >= slots) zero_row<DT>(y + r * cols, cols, lane);
}

// One wave a token and 64 * kGatherPieces pieces of its columns, which it
// writes to the rows of all its choices. Bound by bytes: each token's row is
// read once, each sorted row written once.
constexpr uint32_t kGatherPieces = 1;
template <int DT>
__global__ __launch_bounds__(kRowThreads) void k_expert_gather(const typename Elem<DT>::type *__restrict__ x,
                                                               const int32_t *__restrict__ slot_rows,
                                                               const int32_t *__restrict__ row_slots, uint32_t tokens,
                                                               uint32_t topk, uint32_t cols, uint32_t rows, uint32_t strips,
                                                               typename Elem<DT>::type *__restrict__ y) {
  constexpr uint32_t per = Elem<DT>::per;
  const uint32_t lane = threadIdx.x % kWave;
  const uint64_t unit = static_cast<uint64_t>(block_of_long_grid()) * kRowWaves + wave_index(), units = static_cast<uint64_t>(tokens) * strips;
  if (unit >= units) {
    clear_padding<DT>(y, row_slots, (unit - units) * kPadRows, tokens * topk, cols, rows, lane);
    return;
  }
  const uint32_t token = static_cast<uint32_t>(unit / strips), strip = static_cast<uint32_t>(unit % strips);
  const int32_t *at = slot_rows + static_cast<uint64_t>(token) * topk;
  const typename Elem<DT>::type *src = x + static_cast<uint64_t>(token) * cols;
  const uint32_t c0 = (strip * kGatherPieces * kWave + lane) * per;
  piece_t v[kGatherPieces];
  typename Elem<DT>::type rest[per];
#pragma unroll
  for (uint32_t i = 0; i < kGatherPieces; ++i) {
    const uint32_t c = c0 + i * kWave * per;
    if (c + per <= cols) v[i] = *reinterpret_cast<const piece_t *>(src + c);
    else for (uint32_t q = 0; q < per; ++q) if (c + q < cols) rest[q] = src[c + q];  // one lane's, at most
  }
  for (uint32_t j = 0; j < topk; ++j) {
    const uint32_t row = static_cast<uint32_t>(at[j]);
    if (row >= rows) continue;
    typename Elem<DT>::type *dst = y + static_cast<uint64_t>(row) * cols;
#pragma unroll
    for (uint32_t i = 0; i < kGatherPieces; ++i) {
      const uint32_t c = c0 + i * kWave * per;
      if (c + per <= cols) put(dst + c, v[i]);
      else for (uint32_t q = 0; q < per; ++q) if (c + q < cols) dst[c + q] = rest[q];
    }
  }
}

// One wave a token and 64 pieces of its columns: the rows of its choices,
// four loads in flight, are summed in binary32 and rounded once.
template <int DT>
__global__ __launch_bounds__(kRowThreads) void k_expert_combine(const typename Elem<DT>::type *__restrict__ y,
                                                                const int32_t *__restrict__ slot_rows,
                                                                const float *__restrict__ w, uint32_t tokens,
                                                                uint32_t topk, uint32_t cols, uint32_t rows,
                                                                uint32_t strips, typename Elem<DT>::type *__restrict__ out) {
  constexpr uint32_t per = Elem<DT>::per;
  const uint32_t lane = threadIdx.x % kWave;
  const uint64_t unit = static_cast<uint64_t>(block_of_long_grid()) * kRowWaves + wave_index();
  const uint32_t token = static_cast<uint32_t>(unit / strips), strip = static_cast<uint32_t>(unit % strips);
  if (token >= tokens) return;
  const int32_t *at = slot_rows + static_cast<uint64_t>(token) * topk;
  const float *wt = w ? w + static_cast<uint64_t>(token) * topk : nullptr;
  const uint32_t c = (strip * kWave + lane) * per;
  if (c >= cols) return;
  typename Elem<DT>::type *dst = out + static_cast<uint64_t>(token) * cols + c;
  if (c + per <= cols) {
    float acc[per] = {};
    for (uint32_t j0 = 0; j0 < topk; j0 += 8) {
      piece_t v[8];
      float f[8];
#pragma unroll
      for (uint32_t i = 0; i < 8; ++i) {
        const uint32_t row = j0 + i < topk ? static_cast<uint32_t>(at[j0 + i]) : rows;
        f[i] = row < rows ? (wt ? wt[j0 + i] : 1.0f) : 0.0f;
        v[i] = piece_t{0, 0, 0, 0};
        if (row < rows) v[i] = take(y + static_cast<uint64_t>(row) * cols + c);
        else f[i] = 0.0f;
      }
#pragma unroll
      for (uint32_t i = 0; i < 8; ++i) {
        float e[per];
        Elem<DT>::unpack(v[i], e);
#pragma unroll
        for (uint32_t q = 0; q < per; ++q) acc[q] = __builtin_fmaf(f[i], e[q], acc[q]);
      }
    }
    *reinterpret_cast<piece_t *>(dst) = Elem<DT>::pack(acc);
  } else {
    for (uint32_t q = 0; c + q < cols; ++q) {
      float acc = 0.0f;
      for (uint32_t j = 0; j < topk; ++j) {
        const uint32_t row = static_cast<uint32_t>(at[j]);
        if (row < rows) acc = __builtin_fmaf(wt ? wt[j] : 1.0f, Elem<DT>::load(y + static_cast<uint64_t>(row) * cols + c + q), acc);
      }
      Elem<DT>::store(dst + q, acc);
    }
  }
}

// Combine's gradients: one wave a slot reads dout's row and y's row, writes
// dy's row and the slot's dot product (so dout's row is read topk times, by
// neighbouring waves); the waves past the slots clear the padding rows of dy.
template <int DT>
__global__ __launch_bounds__(kRowThreads) void k_expert_combine_grad(
    const typename Elem<DT>::type *__restrict__ dout, const typename Elem<DT>::type *__restrict__ y,
    const int32_t *__restrict__ slot_rows, const int32_t *__restrict__ row_slots, const float *__restrict__ w,
    uint32_t slots, uint32_t topk, uint32_t cols, uint32_t rows, typename Elem<DT>::type *__restrict__ dy,
    float *__restrict__ dw) {
  constexpr uint32_t per = Elem<DT>::per;
  const uint32_t lane = threadIdx.x % kWave;
  const uint64_t unit = static_cast<uint64_t>(block_of_long_grid()) * kRowWaves + wave_index();
  if (unit >= slots) {
    clear_padding<DT>(dy, row_slots, (unit - slots) * kPadRows, slots, cols, rows, lane);
    return;
  }
  const uint32_t slot = static_cast<uint32_t>(unit);
  const uint32_t row = static_cast<uint32_t>(slot_rows[slot]);
  if (row >= rows) {
    if (lane == 0) dw[slot] = 0.0f;
    return;
  }
  const float wt = w[slot];
  const typename Elem<DT>::type *g = dout + static_cast<uint64_t>(slot / topk) * cols;
  const typename Elem<DT>::type *v = y + static_cast<uint64_t>(row) * cols;
  typename Elem<DT>::type *dst = dy + static_cast<uint64_t>(row) * cols;
  float dot = 0.0f;
#pragma unroll 2
  for (uint32_t c = lane * per; c + per <= cols; c += kWave * per) {
    float a[per], b[per];
    Elem<DT>::unpack(*reinterpret_cast<const piece_t *>(g + c), a);
    Elem<DT>::unpack(take(v + c), b);
#pragma unroll
    for (uint32_t q = 0; q < per; ++q) {
      dot = __builtin_fmaf(a[q], b[q], dot);
      a[q] *= wt;
    }
    put(dst + c, Elem<DT>::pack(a));
  }
  for (uint32_t c = cols / per * per + lane; c < cols; c += kWave) {
    const float a = Elem<DT>::load(g + c);
    dot = __builtin_fmaf(a, Elem<DT>::load(v + c), dot);
    Elem<DT>::store(dst + c, a * wt);
  }
#pragma unroll
  for (uint32_t d = kWave / 2; d > 0; d /= 2) dot += __shfl_xor(dot, d);
  if (lane == 0) dw[slot] = dot;
}

// Slots of a workgroup: one round of its waves, or more where that would
// make over kSortChunks workgroups. (65536 slots, 64 experts: 17.4 us in 16
// workgroups of four rounds, 9.6 us in 64.)
uint64_t sort_chunk(uint64_t slots) {
  const uint64_t c = (slots + kSortChunks - 1) / kSortChunks;
  return (c + kSortThreads - 1) / kSortThreads * kSortThreads;
}

uint64_t blocks_of(uint64_t units, uint64_t per) { return (units + per - 1) / per; }

}  // namespace

uint64_t expert_sort_workspace_words(uint64_t slots, uint32_t experts) {
  return slots <= kSortTile ? 0 : blocks_of(slots, sort_chunk(slots)) * experts;
}

hipError_t launch_expert_sort(const ExpertSort &p, hipStream_t s) {
  SortArgs a{};
  a.ids = p.ids;
  a.wide = p.wide;
  a.slots = p.slots;
  a.experts = p.experts;
  a.align_log2 = p.align_log2;
  a.rows = p.rows;
  a.slot_rows = p.slot_rows;
  a.row_slots = p.row_slots;
  a.offsets = p.offsets;
  a.counts = p.counts;
  a.chunk = p.slots > kSortTile ? static_cast<uint32_t>(sort_chunk(p.slots)) : kSortTile;
  a.chunks = p.slots > kSortTile ? static_cast<uint32_t>(blocks_of(p.slots, a.chunk)) : 1;
  a.rounds = static_cast<uint32_t>(std::min<uint64_t>(kSortRounds, std::max<uint64_t>(1, blocks_of(std::min(p.slots, a.chunk), kSortThreads))));
  a.hist = a.chunks > 1 ? p.workspace : nullptr;
  if (a.chunks > 1) {
    hipLaunchKernelGGL(k_expert_count, dim3(a.chunks), dim3(kSortThreads), 0, s, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(k_expert_place, dim3(a.chunks), dim3(kSortThreads), 0, s, a);
  return hipGetLastError();
}

template <int DT>
static hipError_t gather_t(const ExpertRows &p, hipStream_t s) {
  typedef typename Elem<DT>::type T;
  const uint32_t strips = static_cast<uint32_t>(blocks_of(p.cols, kGatherPieces * kWave * Elem<DT>::per));
  const uint64_t units = static_cast<uint64_t>(p.tokens) * strips + blocks_of(p.rows, kPadRows);
  hipLaunchKernelGGL((k_expert_gather<DT>), long_grid(blocks_of(units, kRowWaves)), dim3(kRowThreads), 0, s,
                     static_cast<const T *>(p.x), p.slot_rows, p.row_slots, p.tokens, p.topk, p.cols, p.rows, strips,
                     static_cast<T *>(p.out));
  return hipGetLastError();
}

template <int DT>
static hipError_t combine_t(const ExpertRows &p, hipStream_t s) {
  typedef typename Elem<DT>::type T;
  const uint32_t strips = static_cast<uint32_t>(blocks_of(p.cols, kWave * Elem<DT>::per));
  const uint64_t blocks = blocks_of(static_cast<uint64_t>(p.tokens) * strips, kRowWaves);
  hipLaunchKernelGGL((k_expert_combine<DT>), long_grid(blocks), dim3(kRowThreads), 0, s,
                     static_cast<const T *>(p.x), p.slot_rows, p.weights, p.tokens, p.topk, p.cols, p.rows, strips,
                     static_cast<T *>(p.out));
  return hipGetLastError();
}

template <int DT>
static hipError_t combine_grad_t(const ExpertRows &p, hipStream_t s) {
  typedef typename Elem<DT>::type T;
  const uint64_t units = static_cast<uint64_t>(p.tokens) * p.topk + blocks_of(p.rows, kPadRows);
  hipLaunchKernelGGL((k_expert_combine_grad<DT>), long_grid(blocks_of(units, kRowWaves)), dim3(kRowThreads), 0,
                     s, static_cast<const T *>(p.x), static_cast<const T *>(p.y), p.slot_rows, p.row_slots, p.weights,
                     p.tokens * p.topk, p.topk, p.cols, p.rows, static_cast<T *>(p.out), p.dweights);
  return hipGetLastError();
}

hipError_t launch_expert_gather(const ExpertRows &p, int dtype, hipStream_t s) {
  return dtype == kBF16 ? gather_t<kBF16>(p, s) : gather_t<kFP32>(p, s);
}

hipError_t launch_expert_combine(const ExpertRows &p, int dtype, hipStream_t s) {
  return dtype == kBF16 ? combine_t<kBF16>(p, s) : combine_t<kFP32>(p, s);
}

hipError_t launch_expert_combine_grad(const ExpertRows &p, int dtype, hipStream_t s) {
  return dtype == kBF16 ? combine_grad_t<kBF16>(p, s) : combine_grad_t<kFP32>(p, s);
}

}  // namespace nvfp4
