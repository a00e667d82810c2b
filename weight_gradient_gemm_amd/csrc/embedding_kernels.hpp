// The embedding: lookup with scaling, and its gradient by sorted tokens.
//
//   out[t] = scale table[ids[t]]
//   g[r]   = scale sum_{t: ids[t] = r} dY[t]
//
// The gradient needs, for every row, its tokens in a fixed order. The token
// positions are sorted by id, stably (a radix sort, so that no distribution of
// ids is slow), the rows' bounds in the sorted order are found by bisection,
// and one pass over the rows sums each row's tokens in registers and stores
// the gradient or steps the optimizer at once. Ids outside [0, V) get the key
// V and end up behind the last row.
//
// Frequent ids: the sorted order is cut into chunks of C = 32 tokens (128 or
// 256 of many: see embedding_chunk_bits). A chunk that lies within one row is summed beforehand by workgroups of its
// own; the row's pass then adds such sums, and the tokens before and after
// them, in ascending order. A row of n tokens costs its pass at most
// 2 (C - 1) + n / C additions in a row, and the order of
// additions depends on the ids alone. Up to kRankTokens tokens a token's place
// is counted instead (rank_kernel), up to kScanTokens nothing is sorted
// (embedding_scan_kernel).
//
// No atomics: a wave ranks its 64 keys with ballots (lanes of equal digit),
// and the lowest lane of each group advances the wave's own counter.
#pragma once

#include <hip/hip_runtime.h>

#include "row_units.hpp"
#include "wgrad_kernels.hpp"

namespace forge {

constexpr int kDigitBits = 9;                        // largest digit of a pass
constexpr int kDigits = 1 << kDigitBits;
constexpr int kRankTokens = 8192;                   // tokens that are ranked by comparing all pairs
constexpr int kRankKeys = 32;                        // of a workgroup then, 8 threads to a key
constexpr int kTileThreads = 256;                    // a tile of the larger sort
constexpr int kTileR = 4;                            // keys of a thread
constexpr int kTileKeys = kTileThreads * kTileR;
constexpr int kDirectTiles = 64;                     // tiles that sum their counts themselves
constexpr int kScanTokens = 256;                     // tokens that are looked through, not sorted
constexpr int kScanUnits = 4;                        // most 256-unit pieces of a workgroup then
constexpr int kScanRows = kScanUnits * 256 / 2 + 1;  // and rows: two units or more, cut at both ends

struct IdSource {
  const void* ids;
  int32_t bytes;       // 4 or 8
  uint32_t V;
};

__device__ __forceinline__ int64_t load_id(const IdSource& src, int64_t t) {
  return src.bytes == 8 ? static_cast<const int64_t*>(src.ids)[t]
                        : int64_t(static_cast<const int32_t*>(src.ids)[t]);
}

// Sort key of token t: its row, or V for nobody's.
__device__ __forceinline__ uint32_t load_key(const IdSource& src, int64_t t) {
  const int64_t id = load_id(src, t);
  return id >= 0 && id < int64_t(src.V) ? uint32_t(id) : src.V;
}

// Sort keys of the tokens first, first + step, ... (N of them), ~0 past the
// last: all loads in flight at once, behind one look at the ids' type.
template <int N>
__device__ __forceinline__ void load_keys(const IdSource& src, int64_t first, int64_t step, int64_t T,
                                          uint32_t (&key)[N]) {
  int64_t id[N];
  if (src.bytes == 8) {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int64_t t = first + j * step;
      id[j] = static_cast<const int64_t*>(src.ids)[t < T ? t : T - 1];
    }
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int64_t t = first + j * step;
      id[j] = static_cast<const int32_t*>(src.ids)[t < T ? t : T - 1];
    }
  }
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const uint32_t k = id[j] >= 0 && id[j] < int64_t(src.V) ? uint32_t(id[j]) : src.V;
    key[j] = first + j * step < T ? k : ~0u;
  }
}

// Lanes of this wave whose digit equals this lane's.
__device__ __forceinline__ uint64_t match_digit(uint32_t digit, int bits) {
  uint64_t m = ~uint64_t(0);
  for (int b = 0; b < bits; ++b) {
    const bool one = (digit >> b) & 1;
    const uint64_t v = __ballot(one);
    m &= one ? v : ~v;
  }
  return m;
}

// Memory accesses of the wave's lanes before this point come before those
// after it, in the compiled code as in the source.
__device__ __forceinline__ void wave_order() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_wave_barrier();
  asm volatile("" ::: "memory");
}

template <int WAVES>
struct SortLds {
  uint32_t count[WAVES][kDigits];
  uint32_t wave_total[WAVES];
};

// Ranks this wave's keys, R times 64 in ascending position: rank[j] is the
// number of earlier keys of the wave with the same digit; count[wave] ends as
// the wave's digit counts. The workgroup synchronises before and after.
template <int WAVES, int R>
__device__ __forceinline__ void rank_keys(SortLds<WAVES>& s, const uint32_t (&key)[R], uint32_t (&rank)[R],
                                          int shift, int bits) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  for (int d = lane; d < (1 << bits); d += 64) s.count[wave][d] = 0;
  const uint64_t lower = (uint64_t(1) << lane) - 1;
#pragma unroll
  for (int j = 0; j < R; ++j) {
    const uint32_t digit = (key[j] >> shift) & ((1u << bits) - 1u);
    const uint64_t same = match_digit(digit, bits);
    // One wave's LDS operations complete in order; wave_order() keeps the
    // compiler's order the same.
    wave_order();
    const uint32_t before = s.count[wave][digit];
    wave_order();
    if ((same & lower) == 0) s.count[wave][digit] = before + __popcll(same);
    rank[j] = before + __popcll(same & lower);
  }
}

// Exclusive sum of one value per thread over the workgroup.
__device__ __forceinline__ uint32_t block_exclusive(uint32_t v, uint32_t* wave_total) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  uint32_t inc = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t up = __shfl_up(inc, d);
    if (lane >= d) inc += up;
  }
  if (lane == 63) wave_total[wave] = inc;
  __syncthreads();
  uint32_t base = 0;
  for (int w = 0; w < wave; ++w) base += wave_total[w];
  __syncthreads();
  return base + inc - v;
}

// Turns the waves' counts of digit d into each wave's first place, from `at` on.
template <int WAVES>
__device__ __forceinline__ void place_waves(SortLds<WAVES>& s, int d, uint32_t at) {
  for (int w = 0; w < WAVES; ++w) {
    const uint32_t c = s.count[w][d];
    s.count[w][d] = at;
    at += c;
  }
}

template <int WAVES>
__device__ __forceinline__ uint32_t digit_total(const SortLds<WAVES>& s, int d) {
  uint32_t sum = 0;
  for (int w = 0; w < WAVES; ++w) sum += s.count[w][d];
  return sum;
}

// Up to kRankTokens tokens in one launch: a token's place is the number of
// smaller (key, position) pairs, counted by 8 threads that go through all keys
// in LDS. T^2 comparisons are cheap beside the launches of a radix sort: the
// whole gradient of 1021 tokens into 5003 x 512 takes 14.1 us, with the tiles below
// 23.1; of 4096 21.1 and 28.4; of 8192 into 32000 x 512 35.1 and 35.4.
__global__ __launch_bounds__(8 * kRankKeys) void rank_kernel(IdSource src, int T, uint32_t* keys,
                                                             uint32_t* pos) {
  __shared__ __attribute__((aligned(16))) uint32_t lk[kRankTokens];
  const int tid = threadIdx.x, part = tid & 7;
  const int padded = (T + 31) & ~31;                   // behind the last: larger than any key
  for (int t0 = tid; t0 < padded; t0 += 8 * 8 * kRankKeys) {
    uint32_t k[8];
    load_keys(src, t0, 8 * kRankKeys, T, k);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (t0 + j * 8 * kRankKeys < padded) lk[t0 + j * 8 * kRankKeys] = k[j];
  }
  __syncthreads();
  const int i = int(blockIdx.x) * kRankKeys + (tid >> 3);
  if (i >= T) return;
  const uint32_t key = lk[i];
  const int own = i >> 2;                              // the group of four that holds i
  uint32_t n = 0;
#pragma unroll 4
  for (int v = part; v < padded / 4; v += 8) {
    const u32x4_t k = *reinterpret_cast<const u32x4_t*>(&lk[4 * v]);
    const uint32_t than = v < own ? key + 1u : key;    // equal keys count where they come first
#pragma unroll
    for (int j = 0; j < 4; ++j) n += k[j] < than;
  }
  if (part == (own & 7))
    for (int j = own * 4; j < i; ++j) n += lk[j] == key;
#pragma unroll
  for (int d = 1; d < 8; d <<= 1) n += uint32_t(__shfl_xor(int(n), d));
  if (part == 0) {
    keys[n] = key;
    pos[n] = uint32_t(i);
  }
}

// The larger sort, per pass: the digit counts of tiles of 1024 keys, and the
// scatter. Up to kDirectTiles tiles a tile adds up the counts that precede its
// own itself; beyond, a launch between the two forms the sums. The gradient of
// 16384 tokens into 32000 x 64 takes 34.4 us with the former and 38.3 with the
// latter, of 65536 57.3 and 56.4, of 131072 83 and 76, of 262144 105 and 85.
// keys_in == nullptr: the first pass, from the ids.
struct SortPass {
  IdSource src;
  const uint32_t *keys_in, *pos_in;
  uint32_t *keys_out, *pos_out;
  uint32_t* count;     // direct: [tiles][kDigits]; else [digits][tiles]
  uint32_t* total;     // else: of each digit
  int64_t T;
  int32_t tiles, shift, bits;
};

__device__ __forceinline__ void load_tile(const SortPass& a, uint32_t (&key)[kTileR], uint32_t (&p)[kTileR]) {
  constexpr int R = kTileR;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t first = int64_t(blockIdx.x) * kTileKeys + wave * R * 64 + lane;
  if (!a.keys_in) {
    load_keys(a.src, first, 64, a.T, key);
#pragma unroll
    for (int j = 0; j < R; ++j) p[j] = uint32_t(first + j * 64);
    return;
  }
#pragma unroll
  for (int j = 0; j < R; ++j) {
    const int64_t t = first + j * 64 < a.T ? first + j * 64 : a.T - 1;
    key[j] = a.keys_in[t];
    p[j] = a.pos_in[t];
  }
#pragma unroll
  for (int j = 0; j < R; ++j)
    if (first + j * 64 >= a.T) key[j] = ~0u;
}

template <bool DIRECT>
__global__ __launch_bounds__(kTileThreads) void sort_count_kernel(SortPass a) {
  __shared__ SortLds<kTileThreads / 64> s;
  uint32_t key[kTileR], p[kTileR], rank[kTileR];
  load_tile(a, key, p);
  rank_keys(s, key, rank, a.shift, a.bits);
  __syncthreads();
  for (int d = threadIdx.x; d < (1 << a.bits); d += kTileThreads) {
    const int64_t at = DIRECT ? int64_t(blockIdx.x) * kDigits + d : int64_t(d) * a.tiles + blockIdx.x;
    a.count[at] = digit_total(s, d);
  }
}

// A digit's counts over the tiles, by a workgroup: their exclusive sums, in place,
// and the digit's total.
__global__ __launch_bounds__(kTileThreads) void sort_sum_kernel(SortPass a) {
  __shared__ uint32_t wave_total[kTileThreads / 64];
  uint32_t* const count = a.count + int64_t(blockIdx.x) * a.tiles;
  uint32_t carry = 0;
  for (int k = 0; k < a.tiles; k += kTileThreads) {
    const int at = k + int(threadIdx.x);
    const uint32_t v = at < a.tiles ? count[at] : 0;
    const uint32_t before = carry + block_exclusive(v, wave_total);
    for (int w = 0; w < kTileThreads / 64; ++w) carry += wave_total[w];
    __syncthreads();
    if (at < a.tiles) count[at] = before;
  }
  if (threadIdx.x == 0) a.total[blockIdx.x] = carry;
}

template <bool DIRECT>
__global__ __launch_bounds__(kTileThreads) void sort_scatter_kernel(SortPass a) {
  __shared__ SortLds<kTileThreads / 64> s;
  uint32_t key[kTileR], p[kTileR], rank[kTileR];
  load_tile(a, key, p);
  rank_keys(s, key, rank, a.shift, a.bits);
  __syncthreads();
  // A thread takes the digits 2 t and 2 t + 1.
  static_assert(kDigits == 2 * kTileThreads, "two digits to a thread");
  const int d = 2 * int(threadIdx.x);
  const bool mine = d < (1 << a.bits);     // bits >= 1: both digits or none
  uint32_t at[2] = {0u, 0u}, total[2] = {0u, 0u};
  if constexpr (DIRECT) {
    if (mine) {
#pragma unroll 8
      for (int t = 0; t < a.tiles; ++t) {
        const u32x2_t c = *reinterpret_cast<const u32x2_t*>(a.count + int64_t(t) * kDigits + d);
        total[0] += c[0];
        total[1] += c[1];
        if (t < int(blockIdx.x)) {
          at[0] += c[0];
          at[1] += c[1];
        }
      }
    }
  } else if (mine) {
    for (int k = 0; k < 2; ++k) {
      total[k] = a.total[d + k];
      at[k] = a.count[int64_t(d + k) * a.tiles + blockIdx.x];
    }
  }
  const uint32_t base = block_exclusive(total[0] + total[1], s.wave_total);
  at[0] += base;
  at[1] += base + total[0];
  if (mine) {
    place_waves(s, d, at[0]);
    place_waves(s, d + 1, at[1]);
  }
  __syncthreads();
  const int wave = threadIdx.x >> 6;
#pragma unroll
  for (int j = 0; j < kTileR; ++j) {
    const uint32_t to = s.count[wave][(key[j] >> a.shift) & ((1u << a.bits) - 1u)] + rank[j];
    if (int64_t(to) < a.T) {       // keys past the last token come last
      a.keys_out[to] = key[j];
      a.pos_out[to] = p[j];
    }
  }
}

struct EmbeddingArgs {
  const uint32_t *keys, *pos;      // sorted
  uint32_t* bound;                 // [V + 1]: first sorted place of each row
  float* chunk;                    // [T >> chunk_bits, d]: sums of chunks within one row
  const void* dY;
  float *W, *m, *v;                // W: the gradient, where it is stored
  int64_t T;
  int32_t V, d, chunk_bits;
  Rows rows;                       // of 4-column units
  uint32_t slices;                 // 1024-column slices of a row (chunk sums)
  uint32_t bound_blocks;           // workgroups of the bounds kernel that search
  uint32_t blocks;                 // workgroups of a pass (a launch may have fewer, and loop)
  uint32_t scan_units;             // 256-unit pieces of a workgroup that looks through the ids
  float scale;
  AdamWConsts adam;
  SgdmConsts sgd;
};

template <bool BF16>
__device__ __forceinline__ f32x4_t load_dy4(const void* dY, int64_t i) {
  if constexpr (BF16)
    return __builtin_convertvector(
        *reinterpret_cast<const bf16x4_t*>(static_cast<const __bf16*>(dY) + i), f32x4_t);
  else
    return *reinterpret_cast<const f32x4_t*>(static_cast<const float*>(dY) + i);
}

// acc += term(s) + ... + term(e - 1), one after the other. Loads go U at a
// time, the last ones four at a time, where places past the end repeat the last
// term and are not added. U costs registers: 8 where a row is only written (V
// 128256 x 512, 1025 tokens: 49 us against 74 with 16), 16 where it is stepped
// (AdamW, 16384 tokens into 32000 x 1024: 151 us against 157 with 8; into 128256 x
// 4096 runs differ by more, 2.05-2.20 ms with either).
template <int U, class Term>
__device__ __forceinline__ void add_terms(f32x4_t& acc, uint32_t s, uint32_t e, const Term& term) {
  for (; s + U <= e; s += U) {
    f32x4_t r[U];
#pragma unroll
    for (int j = 0; j < U; ++j) r[j] = term(s + j);
#pragma unroll
    for (int j = 0; j < U; ++j) acc = acc + r[j];
  }
  for (; s < e; s += 4) {
    f32x4_t r[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) r[j] = term(s + j < e ? s + j : e - 1);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const f32x4_t sum = acc + r[j];
      acc = s + j < e ? sum : acc;
    }
  }
}

// acc += the tokens at sorted places [s, e).
template <int U, bool BF16>
__device__ __forceinline__ void add_tokens(const EmbeddingArgs& a, f32x4_t& acc, uint32_t s,
                                           uint32_t e, int col) {
  add_terms<U>(acc, s, e, [&](uint32_t k) {
    return load_dy4<BF16>(a.dY, int64_t(a.pos[k]) * a.d + col);
  });
}

// The rows' bounds (the first workgroups, one row per thread), and the sums of
// the chunks that lie within one row (the others, one slice of a chunk each).
template <bool BF16>
__global__ __launch_bounds__(256) void embedding_bounds_kernel(EmbeddingArgs a) {
  for (uint32_t b = blockIdx.x; b < a.blocks; b += gridDim.x) {
    if (b < a.bound_blocks) {
      const uint32_t r = b * 256 + threadIdx.x;
      if (r <= uint32_t(a.V)) {
        uint32_t lo = 0, hi = uint32_t(a.T);       // first place whose key is >= r
        while (lo < hi) {
          const uint32_t mid = lo + (hi - lo) / 2;
          if (a.keys[mid] < r)
            lo = mid + 1;
          else
            hi = mid;
        }
        a.bound[r] = lo;
      }
      continue;
    }
    const uint32_t c = (b - a.bound_blocks) / a.slices, slice = b - a.bound_blocks - c * a.slices;
    const uint32_t s = c << a.chunk_bits, e = s + (1u << a.chunk_bits), key = a.keys[s];
    if (key >= uint32_t(a.V) || a.keys[e - 1] != key) continue;
    const int col = int(slice * 256 + threadIdx.x) * 4;
    if (col < a.d) {
      f32x4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
      add_tokens<16, BF16>(a, acc, s, e, col);
      *reinterpret_cast<f32x4_t*>(a.chunk + int64_t(c) * a.d + col) = acc;
    }
  }
}

enum EmbOp : int { EMB_GRAD = 0, EMB_GRAD_ADD = 1, EMB_ADAMW = 2, EMB_ADAMW_EXACT = 3, EMB_SGDM = 4 };

// One row's gradient g (unscaled) at 4 columns, stored or consumed: `sum(g)`
// adds the row's tokens, after W and the state have been requested. They are
// read and written once: non-temporal, as in the clipped steps.
template <int OP, class Sum>
__device__ __forceinline__ void row_step(const EmbeddingArgs& a, int64_t i, const Sum& sum) {
  constexpr bool ADAM = OP == EMB_ADAMW || OP == EMB_ADAMW_EXACT;
  auto get4 = [](const float* p) {
    return __builtin_nontemporal_load(reinterpret_cast<const f32x4_t*>(p));
  };
  auto set4 = [](float* p, const f32x4_t& x) {
    __builtin_nontemporal_store(x, reinterpret_cast<f32x4_t*>(p));
  };
  f32x4_t w, m, v;
  if constexpr (OP != EMB_GRAD) w = get4(a.W + i);
  if constexpr (ADAM || OP == EMB_SGDM) m = get4(a.m + i);
  if constexpr (ADAM) v = get4(a.v + i);
  f32x4_t g = {0.0f, 0.0f, 0.0f, 0.0f};
  sum(g);
  g = g * a.scale;
  if constexpr (OP == EMB_GRAD) w = g;
  if constexpr (OP == EMB_GRAD_ADD) w = w + g;
  if constexpr (ADAM) adamw_vec4<OP == EMB_ADAMW_EXACT>(g, w, m, v, a.adam);
  if constexpr (OP == EMB_SGDM) sgdm_vec4(g, w, m, a.sgd);
  set4(a.W + i, w);
  if constexpr (ADAM || OP == EMB_SGDM) set4(a.m + i, m);
  if constexpr (ADAM) set4(a.v + i, v);
}

// Waves per SIMD that the rows' passes are compiled for: rows that are only
// written keep to the 64 registers that eight need. (Compiled for 4 or 7 they take
// 64 as well, and the same 327 us for 16384 tokens into 128256 x 4096.)
template <int OP>
constexpr int kRowWaves = OP == EMB_GRAD ? 8 : OP == EMB_GRAD_ADD ? 7 : 4;

// 4 columns of one row per thread.
// 16384 tokens into 128256 x 4096 with AdamW: 2.0-2.2 ms, 12.7 GB (5.9-6.2 TB/s,
// what a stream of reads and writes reaches).
template <int OP, bool BF16>
__global__ __launch_bounds__(256, kRowWaves<OP>) void embedding_rows_kernel(EmbeddingArgs a) {
  constexpr int U = OP == EMB_GRAD || OP == EMB_GRAD_ADD ? 8 : 16;
  for (uint32_t b = blockIdx.x; b < a.blocks; b += gridDim.x) {
    uint32_t row, unit;
    locate(a.rows, uint64_t(b) * 256, threadIdx.x, row, unit);
    if (row >= uint32_t(a.V)) continue;
    const int col = int(unit) * 4;
    const uint32_t s = a.bound[row], e = a.bound[row + 1];
    if (OP == EMB_GRAD_ADD && s == e) continue;
    row_step<OP>(a, int64_t(row) * a.d + col, [&](f32x4_t& g) {
      const uint32_t c0 = (s + (1u << a.chunk_bits) - 1) >> a.chunk_bits, c1 = e >> a.chunk_bits;
      if (c0 < c1) {
        add_tokens<U, BF16>(a, g, s, c0 << a.chunk_bits, col);
        add_terms<U>(g, c0, c1, [&](uint32_t c) {
          return *reinterpret_cast<const f32x4_t*>(a.chunk + int64_t(c) * a.d + col);
        });
        add_tokens<U, BF16>(a, g, c1 << a.chunk_bits, e, col);
      } else {
        add_tokens<U, BF16>(a, g, s, e, col);
      }
    });
  }
}

// Few tokens: no sort. A workgroup takes a.scan_units * 256 units, looks
// through all ids for those of its rows, and lists its rows' tokens in
// ascending order in LDS: one launch instead of three. 255 tokens into 5003 x
// 512: 6.3 us, where the ranking and its successors take 11.4; all of one row: 19.1
// against 12.6, and of 64 tokens 8.2 against 10.7.
template <int OP, bool BF16>
__global__ __launch_bounds__(kScanTokens) void embedding_scan_kernel(EmbeddingArgs a, IdSource src) {
  constexpr int U = OP == EMB_GRAD || OP == EMB_GRAD_ADD ? 8 : 16;
  constexpr int WAVES = kScanTokens / 64;
  static_assert(kScanTokens == 256, "an id to a thread");
  // Found tokens, each with its row in bits 16 and up, and four behind the last.
  __shared__ __attribute__((aligned(16))) uint32_t found[kScanTokens + 4];
  __shared__ uint16_t list[kScanTokens];               // tokens by row, ascending
  __shared__ uint32_t count[WAVES], first[kScanRows + 1];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  for (uint32_t b = blockIdx.x; b < a.blocks; b += gridDim.x) {
    const uint64_t unit0 = uint64_t(b) * a.scan_units * 256;
    uint32_t r0, r1, unit;
    locate(a.rows, unit0, 0, r0, unit);
    locate(a.rows, unit0 + (a.scan_units - 1) * 256, 255, r1, unit);
    const int rows = int(min(r1 + 1, uint32_t(a.V)) - r0);
    // A key of V (nobody's) lies past the last row.
    const uint32_t key = tid < a.T ? load_key(src, tid) - r0 : ~0u;
    const uint64_t mine = __ballot(key < uint32_t(rows));
    if (lane == 0) count[wave] = __popcll(mine);
    __syncthreads();
    uint32_t total = 0, before = 0;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) {
      if (w < wave) before += count[w];
      total += count[w];
    }
    if (total > 0) {
      if (key < uint32_t(rows))
        found[before + __popcll(mine & ((uint64_t(1) << lane) - 1))] = uint32_t(tid) | key << 16;
      if (tid < 4) found[total + tid] = ~0u;
      __syncthreads();
      // An entry's place is the number of smaller ones, a row's first place the
      // number of entries of the rows before it.
      auto smaller = [&](uint32_t than) {
        uint32_t n = 0;
#pragma unroll 4
        for (uint32_t k = 0; k < total; k += 4) {
          const u32x4_t f = *reinterpret_cast<const u32x4_t*>(&found[k]);
#pragma unroll
          for (int j = 0; j < 4; ++j) n += f[j] < than;
        }
        return n;
      };
      if (uint32_t(tid) < total) list[smaller(found[tid])] = uint16_t(found[tid]);
      for (int r = tid; r <= rows; r += 256) first[r] = smaller(uint32_t(r) << 16);
    } else {
      for (int r = tid; r <= rows; r += 256) first[r] = 0;
    }
    __syncthreads();
    for (uint32_t k = 0; k < a.scan_units; ++k) {
      uint32_t row;
      locate(a.rows, unit0 + k * 256, tid, row, unit);
      if (row >= uint32_t(a.V)) break;
      const int col = int(unit) * 4;
      const uint32_t s = first[row - r0], e = first[row - r0 + 1];
      if (OP == EMB_GRAD_ADD && s == e) continue;
      row_step<OP>(a, int64_t(row) * a.d + col, [&](f32x4_t& g) {
        add_terms<U>(g, s, e, [&](uint32_t t) {
          return load_dy4<BF16>(a.dY, int64_t(list[t]) * a.d + col);
        });
      });
    }
    __syncthreads();                                   // the next rows reuse the LDS
  }
}

struct LookupArgs {
  IdSource src;
  const void* table;
  void* out;
  int64_t T;
  int32_t d;
  Rows rows;           // of 8-column units
  uint32_t blocks;
  float scale;
};

// 8 columns of one token per thread. STREAM: stores with the non-temporal hint,
// for outputs that would fill the 256 MB cache anyway. 16384 x 4096 bf16 (134
// MB): 44 us against 47, with a reader behind it 77 against 76; 4096 tokens (34
// MB): 13.4 against 13.8, but with the reader 28.7 against 25.5.
template <bool TABLE_BF16, bool OUT_BF16, bool STREAM>
__global__ __launch_bounds__(256) void embedding_kernel(LookupArgs a) {
  auto put = [](const auto& v, auto* p) {
    if constexpr (STREAM)
      __builtin_nontemporal_store(v, p);
    else
      *p = v;
  };
  for (uint32_t b = blockIdx.x; b < a.blocks; b += gridDim.x) {
    uint32_t t, unit;
    locate(a.rows, uint64_t(b) * 256, threadIdx.x, t, unit);
    if (t >= a.T) continue;
    const int col = int(unit) * 8;
    const uint32_t row = load_key(a.src, t);
    f32x4_t x[2] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
    if (row < a.src.V) {
      const int64_t i = int64_t(row) * a.d + col;
      if constexpr (TABLE_BF16) {
        const u32x4_t raw = *reinterpret_cast<const u32x4_t*>(static_cast<const uint16_t*>(a.table) + i);
        x[0] = unpack_bf16x4(u32x2_t{raw[0], raw[1]});
        x[1] = unpack_bf16x4(u32x2_t{raw[2], raw[3]});
      } else {
        const f32x4_t* p = reinterpret_cast<const f32x4_t*>(static_cast<const float*>(a.table) + i);
        x[0] = p[0];
        x[1] = p[1];
      }
      x[0] = x[0] * a.scale;
      x[1] = x[1] * a.scale;
    }
    const int64_t o = int64_t(t) * a.d + col;
    if constexpr (OUT_BF16) {
      const u32x2_t lo = pack_bf16x4(x[0]), hi = pack_bf16x4(x[1]);
      put(u32x4_t{lo[0], lo[1], hi[0], hi[1]}, reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(a.out) + o));
    } else {
      f32x4_t* p = reinterpret_cast<f32x4_t*>(static_cast<float*>(a.out) + o);
      put(x[0], p);
      put(x[1], p + 1);
    }
  }
}

}  // namespace forge
