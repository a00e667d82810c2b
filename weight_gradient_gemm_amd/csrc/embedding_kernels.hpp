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
// Frequent ids: the sorted order is cut into chunks of kSumChunk tokens. A
// chunk that lies within one row is summed beforehand by workgroups of its
// own; the row's pass then adds such sums, and the tokens before and after
// them, in ascending order. A row of n tokens costs its pass at most
// 2 (kSumChunk - 1) + n / kSumChunk additions in a row, and the order of
// additions depends on the ids alone.
//
// No atomics: a wave ranks its 64 keys with ballots (lanes of equal digit),
// and the lowest lane of each group advances the wave's own counter.
#pragma once

#include <hip/hip_runtime.h>

#include "wgrad_kernels.hpp"

namespace forge {

constexpr int kDigitBits = 9;                        // largest digit of a pass
constexpr int kDigits = 1 << kDigitBits;
constexpr int kOneThreads = 1024;                    // the one-workgroup sort
constexpr int kOneRounds = 4;                        // its keys per thread
constexpr int kSortOne = kOneThreads * kOneRounds;
constexpr int kTileThreads = 256;                    // a tile of the larger sort
constexpr int kDirectTiles = 64;                     // tiles that sum their counts themselves
constexpr int kSumChunk = 32;
constexpr int kScanTokens = 256;                     // tokens that are looked through, not sorted
constexpr int kScanRows = 64;                        // most rows of a workgroup then

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

// Ranks this wave's keys, `rounds` of 64 in ascending position: rank[j] is the
// number of earlier keys of the wave with the same digit; count[wave] ends as
// the wave's digit counts. The workgroup synchronises before and after.
template <int WAVES, int R>
__device__ __forceinline__ void rank_keys(SortLds<WAVES>& s, const uint32_t (&key)[R], uint32_t (&rank)[R],
                                          int rounds, int shift, int bits) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  for (int d = lane; d < (1 << bits); d += 64) s.count[wave][d] = 0;
  const uint64_t lower = (uint64_t(1) << lane) - 1;
#pragma unroll
  for (int j = 0; j < R; ++j) {
    if (j < rounds) {
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

// Up to kSortOne tokens by one workgroup, in LDS (1021 tokens: 7.8 us).
__global__ __launch_bounds__(kOneThreads) void sort_one_kernel(IdSource src, int T, int key_bits,
                                                               uint32_t* keys, uint32_t* pos) {
  constexpr int WAVES = kOneThreads / 64, R = kOneRounds;
  __shared__ SortLds<WAVES> s;
  __shared__ uint32_t lk[kSortOne];
  __shared__ uint16_t lp[kSortOne];
  static_assert(kSortOne <= 65536, "positions are kept in 16 bits");
  static_assert(kDigits <= kOneThreads, "a thread to a digit");
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int rounds = (T + kOneThreads - 1) / kOneThreads;
  const int first = wave * rounds * 64 + lane;
  uint32_t key[R], p[R], rank[R];
#pragma unroll
  for (int j = 0; j < R; ++j) {
    const int t = first + j * 64;
    // Past the last token: behind every key, in every pass.
    key[j] = j < rounds && t < T ? load_key(src, t) : 0xffffffffu;
    p[j] = t;
  }
  const int passes = (key_bits + kDigitBits - 1) / kDigitBits;
  for (int k = 0; k < passes; ++k) {
    const int shift = key_bits * k / passes, bits = key_bits * (k + 1) / passes - shift;
    rank_keys(s, key, rank, rounds, shift, bits);
    __syncthreads();
    const int d = threadIdx.x;
    const bool mine = d < (1 << bits);
    const uint32_t at = block_exclusive(mine ? digit_total(s, d) : 0u, s.wave_total);
    if (mine) place_waves(s, d, at);
    __syncthreads();
    const bool last = k + 1 == passes;
#pragma unroll
    for (int j = 0; j < R; ++j) {
      if (j < rounds) {
        const uint32_t to = s.count[wave][(key[j] >> shift) & ((1u << bits) - 1u)] + rank[j];
        if (!last) {
          lk[to] = key[j];
          lp[to] = uint16_t(p[j]);
        } else if (to < uint32_t(T)) {
          keys[to] = key[j];
          pos[to] = p[j];
        }
      }
    }
    if (!last) {
      __syncthreads();
#pragma unroll
      for (int j = 0; j < R; ++j)
        if (j < rounds) {
          key[j] = lk[first + j * 64];
          p[j] = lp[first + j * 64];
        }
      __syncthreads();
    }
  }
}

// The larger sort, per pass: the digit counts of tiles of 256 R keys, and the
// scatter. Up to kDirectTiles tiles, a tile adds up the counts that precede its
// own itself (one launch less, and the counts come from L2); beyond, a launch
// between the two turns them into places. R is 4 up to 65536 tokens (16384:
// 21 us, where one workgroup took 38) and 16 beyond.
// keys_in == nullptr: the first pass, from the ids.
struct SortPass {
  IdSource src;
  const uint32_t *keys_in, *pos_in;
  uint32_t *keys_out, *pos_out;
  uint32_t* count;     // direct: [tiles][kDigits]; else [digits][tiles]
  int64_t T;
  int32_t tiles, shift, bits;
};

template <int R>
__device__ __forceinline__ void load_tile(const SortPass& a, uint32_t (&key)[R], uint32_t (&p)[R]) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t first = int64_t(blockIdx.x) * (kTileThreads * R) + wave * R * 64 + lane;
#pragma unroll
  for (int j = 0; j < R; ++j) {
    const int64_t t = first + j * 64;
    const bool in = t < a.T;
    key[j] = !in ? 0xffffffffu : a.keys_in ? a.keys_in[t] : load_key(a.src, t);
    p[j] = !in ? 0u : a.keys_in ? a.pos_in[t] : uint32_t(t);
  }
}

template <int R, bool DIRECT>
__global__ __launch_bounds__(kTileThreads) void sort_count_kernel(SortPass a) {
  __shared__ SortLds<kTileThreads / 64> s;
  uint32_t key[R], p[R], rank[R];
  load_tile(a, key, p);
  rank_keys(s, key, rank, R, a.shift, a.bits);
  __syncthreads();
  for (int d = threadIdx.x; d < (1 << a.bits); d += kTileThreads) {
    const int64_t at = DIRECT ? int64_t(blockIdx.x) * kDigits + d : int64_t(d) * a.tiles + blockIdx.x;
    a.count[at] = digit_total(s, d);
  }
}

// Exclusive sum of n counts, in place, by one workgroup.
__global__ __launch_bounds__(kOneThreads) void sort_sum_kernel(uint32_t* count, int64_t n) {
  constexpr int WAVES = kOneThreads / 64, E = 8;
  __shared__ uint32_t wave_total[WAVES];
  uint32_t carry = 0;
  for (int64_t k = 0; k < n; k += kOneThreads * E) {
    uint32_t v[E], sum = 0;
    const int64_t at = k + int64_t(threadIdx.x) * E;
#pragma unroll
    for (int j = 0; j < E; ++j) {
      v[j] = at + j < n ? count[at + j] : 0;
      sum += v[j];
    }
    uint32_t before = carry + block_exclusive(sum, wave_total);
    for (int w = 0; w < WAVES; ++w) carry += wave_total[w];
    __syncthreads();
#pragma unroll
    for (int j = 0; j < E; ++j) {
      if (at + j < n) count[at + j] = before;
      before += v[j];
    }
  }
}

template <int R, bool DIRECT>
__global__ __launch_bounds__(kTileThreads) void sort_scatter_kernel(SortPass a) {
  __shared__ SortLds<kTileThreads / 64> s;
  uint32_t key[R], p[R], rank[R];
  load_tile(a, key, p);
  rank_keys(s, key, rank, R, a.shift, a.bits);
  __syncthreads();
  // A thread takes the digits 2 t and 2 t + 1.
  static_assert(kDigits == 2 * kTileThreads, "two digits to a thread");
  const int d = 2 * int(threadIdx.x);
  const bool mine = d < (1 << a.bits);     // bits >= 1: both digits or none
  uint32_t at[2] = {0u, 0u};
  if constexpr (DIRECT) {
    uint32_t total[2] = {0u, 0u};
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
    const uint32_t base = block_exclusive(total[0] + total[1], s.wave_total);
    at[0] += base;
    at[1] += base + total[0];
  } else if (mine) {
    at[0] = a.count[int64_t(d) * a.tiles + blockIdx.x];
    at[1] = a.count[int64_t(d + 1) * a.tiles + blockIdx.x];
  }
  if (mine) {
    place_waves(s, d, at[0]);
    place_waves(s, d + 1, at[1]);
  }
  __syncthreads();
  const int wave = threadIdx.x >> 6;
#pragma unroll
  for (int j = 0; j < R; ++j) {
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
  float* chunk;                    // [T / kSumChunk, d]: sums of chunks within one row
  const void* dY;
  float *W, *m, *v;                // W: the gradient, where it is stored
  int64_t T;
  int32_t V, d;
  int32_t lanes_log2;              // threads across a row in a workgroup
  uint32_t slices;                 // workgroups across a row
  uint32_t bound_blocks;           // workgroups of the bounds kernel that search
  uint32_t blocks;                 // workgroups of a pass (a launch may have fewer, and loop)
  int32_t scan_rows;               // rows of a workgroup that looks through the ids
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
// 128256 x 512, 1025 tokens: 50 us against 65 with 16), 16 where it is read too
// (AdamW, 128256 x 4096: 2.15 ms against 2.22 with 8).
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
    const uint32_t s = c * kSumChunk, key = a.keys[s];
    if (key >= uint32_t(a.V) || a.keys[s + kSumChunk - 1] != key) continue;
    const int col = int(slice * 256 + threadIdx.x) * 4;
    if (col < a.d) {
      f32x4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
      add_tokens<16, BF16>(a, acc, s, s + kSumChunk, col);
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

// One row (or several short ones) per workgroup, 4 columns per thread.
// 16384 tokens into 128256 x 4096 with AdamW: 2.2 ms, 12.7 GB (5.8 TB/s, what a
// stream of reads and writes reaches).
template <int OP, bool BF16>
__global__ __launch_bounds__(256) void embedding_rows_kernel(EmbeddingArgs a) {
  constexpr int U = OP == EMB_GRAD || OP == EMB_GRAD_ADD ? 8 : 16;
  const int lanes = 1 << a.lanes_log2;
  for (uint32_t b = blockIdx.x; b < a.blocks; b += gridDim.x) {
    const uint32_t rb = b / a.slices, slice = b - rb * a.slices;
    const int row = int((rb << (8 - a.lanes_log2)) + (threadIdx.x >> a.lanes_log2));
    const int col = (int(slice << a.lanes_log2) + (int(threadIdx.x) & (lanes - 1))) * 4;
    if (row >= a.V || col >= a.d) continue;
    const uint32_t s = a.bound[row], e = a.bound[row + 1];
    if (OP == EMB_GRAD_ADD && s == e) continue;
    row_step<OP>(a, int64_t(row) * a.d + col, [&](f32x4_t& g) {
      const uint32_t c0 = (s + kSumChunk - 1) / kSumChunk, c1 = e / kSumChunk;
      if (c0 < c1) {
        add_tokens<U, BF16>(a, g, s, c0 * kSumChunk, col);
        add_terms<U>(g, c0, c1, [&](uint32_t c) {
          return *reinterpret_cast<const f32x4_t*>(a.chunk + int64_t(c) * a.d + col);
        });
        add_tokens<U, BF16>(a, g, c1 * kSumChunk, e, col);
      } else {
        add_tokens<U, BF16>(a, g, s, e, col);
      }
    });
  }
}

// Few tokens: no sort. A workgroup takes a.scan_rows rows of one slice of
// columns, looks through all ids for its own, and lists its rows' tokens in
// ascending order in LDS: one launch instead of three. 256 tokens into 5003 x
// 512: 5.7 us, where the sort and its successors take 13.3 for 257; all of one
// row: 16.4 against 11.6. With the limit at 1024 the latter were 94 against 14.
template <int OP, bool BF16>
__global__ __launch_bounds__(kScanTokens) void embedding_scan_kernel(EmbeddingArgs a, IdSource src) {
  constexpr int U = OP == EMB_GRAD || OP == EMB_GRAD_ADD ? 8 : 16;
  constexpr int WAVES = kScanTokens / 64;
  // Found tokens, each with its row in bits 16 and up, and four behind the last.
  __shared__ __attribute__((aligned(16))) uint32_t found[kScanTokens + 4];
  __shared__ uint16_t list[kScanTokens];               // tokens by row, ascending
  __shared__ uint32_t count[WAVES], first[kScanRows + 1];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  for (uint32_t b = blockIdx.x; b < a.blocks; b += gridDim.x) {
    const uint32_t rb = b / a.slices, slice = b - rb * a.slices;
    const uint32_t r0 = rb * uint32_t(a.scan_rows);
    const int rows = int(min(uint32_t(a.V) - r0, uint32_t(a.scan_rows)));
    // A key of V (nobody's) lies past the last row's workgroup.
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
      if (tid <= rows) first[tid] = smaller(uint32_t(tid) << 16);
    } else if (tid <= rows) {
      first[tid] = 0;
    }
    __syncthreads();
    const int lanes = 1 << a.lanes_log2;
    const int col = (int(slice << a.lanes_log2) + (tid & (lanes - 1))) * 4;
    if (col < a.d)
      for (int r = tid >> a.lanes_log2; r < rows; r += 256 >> a.lanes_log2) {
        const uint32_t s = first[r], e = first[r + 1];
        if (OP == EMB_GRAD_ADD && s == e) continue;
        row_step<OP>(a, (int64_t(r0) + r) * a.d + col, [&](f32x4_t& g) {
          add_terms<U>(g, s, e, [&](uint32_t k) {
            return load_dy4<BF16>(a.dY, int64_t(list[k]) * a.d + col);
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
  int32_t d, lanes_log2;
  uint32_t slices, blocks;
  float scale;
};

// 8 columns of one token per thread. STREAM: stores with the non-temporal hint,
// for outputs that would fill the 256 MB cache anyway. 16384 x 4096 bf16 (134
// MB): 45 us against 52, with a reader behind it 76 against 75; 4096 tokens (34
// MB): 13.0 against 14.2, and 22.6 against 22.3.
template <bool TABLE_BF16, bool OUT_BF16, bool STREAM>
__global__ __launch_bounds__(256) void embedding_kernel(LookupArgs a) {
  auto put = [](const auto& v, auto* p) {
    if constexpr (STREAM)
      __builtin_nontemporal_store(v, p);
    else
      *p = v;
  };
  const int lanes = 1 << a.lanes_log2;
  for (uint32_t b = blockIdx.x; b < a.blocks; b += gridDim.x) {
    const uint32_t rb = b / a.slices, slice = b - rb * a.slices;
    const int64_t t = (rb << (8 - a.lanes_log2)) + (threadIdx.x >> a.lanes_log2);
    const int col = (int(slice << a.lanes_log2) + (int(threadIdx.x) & (lanes - 1))) * 8;
    if (t >= a.T || col >= a.d) continue;
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
    const int64_t o = t * a.d + col;
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
