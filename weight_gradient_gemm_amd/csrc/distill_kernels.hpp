// Distillation from a teacher's top logits for gfx950: each row's loss and the
// gradient of the student's logits.
//
//   q = softmax(u / tau) over the row's entries, p = softmax(z / tau) over V columns
//   loss = scale w tau^2 sum_j q_j (log q_j - log p[id_j])
//   dz_i = scale w tau (p_i - sum of the q_j with id_j == i)
//
// Bound by HBM: the logits are read and the gradient is written. Of many rows a
// workgroup takes one after the other and holds it in registers, 16 vectors of 16
// bytes to a thread (a row of 128256 bf16 logits is 250 KB, a CU's registers hold
// 512), so that it is read once, and the next row's vectors are requested as this
// one's leave. What is beyond the registers (65536 float32 columns) is read again for
// the gradient. Few rows are cut into chunks, a workgroup each: one launch forms
// each chunk's maximum and sum of exponentials, a second joins them and forms the
// gradient. The loss alone goes once through a row and holds nothing.
//
// Measured: 4096 x 128256 bf16, a row in 8 left out, 411 us for 1.97 GB, 4.8 TB/s, what
// a copy reaches; 1021 x 32003 float32 with a bf16 gradient 43 us, 4.2 TB/s of the needed
// bytes (entries' columns are written twice); 1024 x 128256 float32, not held whole, 206
// us for the 1.05 GB that it cannot do without and 0.26 again; the loss of 511 x 50021
// float32 17 us, 5.3 TB/s; 8 x 128256 bf16 7.6 us in a graph (traced alone 3.3 and 5.1), two
// launches that wait for memory two and one time. A row read twice by the same grid, the
// maximum first, took 1642 us for the first of these.
//
// The teacher's columns are written with the others and once more, with their q,
// behind a barrier: the workgroup that has the column does both.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "row_io.hpp"

namespace forge {

typedef int i32x4_t __attribute__((ext_vector_type(4)));

constexpr int kDistillMaxK = 1024;

struct DistillArgs {
  const void *z, *teacher, *ids;
  const float* weight;               // NULL: 1
  float* loss;
  void* grad;                        // NULL: the loss alone
  float2* stats;                     // [T][chunks]: maximum, sum of 2^((z - maximum) c)
  float* logit;                      // [T][K]: the student's logit of each entry
  int64_t T, ld, items;              // items: rows times chunks of the launch, one to a workgroup
  int32_t V, K, chunks, chunks_out;  // chunks of V and of ld columns
  int32_t wide_ids, teacher_bf16;
  float c, loss_scale, grad_scale;   // log2(e) / tau, scale tau^2, scale tau
};

// A row's entries: id (-1: not there), 2^((u - largest) c), the student's logit.
struct Entries {
  int32_t id[kDistillMaxK];
  float q[kDistillMaxK];
  float z[kDistillMaxK];
};

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

__device__ __forceinline__ int64_t entry_id(const DistillArgs& a, int64_t at) {
  return a.wide_ids ? static_cast<const int64_t*>(a.ids)[at] : int64_t(static_cast<const int32_t*>(a.ids)[at]);
}
__device__ __forceinline__ float entry_logit(const DistillArgs& a, int64_t at) {
  return a.teacher_bf16 ? __builtin_bit_cast(float, uint32_t(static_cast<const uint16_t*>(a.teacher)[at]) << 16)
                        : static_cast<const float*>(a.teacher)[at];
}
template <bool ZB>
__device__ __forceinline__ float student_logit(const DistillArgs& a, int64_t at) {
  return ZB ? __builtin_bit_cast(float, uint32_t(static_cast<const uint16_t*>(a.z)[at]) << 16)
            : static_cast<const float*>(a.z)[at];
}

// The value that stands for a maximum in differences: 0 where everything is
// -infinity, so that a difference is -infinity and no NaN. What is scaled from one
// maximum to a larger one keeps its own as it is: a sum of nothing times 2^-infinity.
__device__ __forceinline__ float finite_max(float m) { return m == -INFINITY ? 0.0f : m; }

// A vector of 16 bytes of a row and its elements.
template <bool ZB>
constexpr int kVec = ZB ? 8 : 4;
template <bool ZB>
__device__ __forceinline__ void unpack(const u32x4_t& r, float (&v)[kVec<ZB>]) {
#pragma unroll
  for (int k = 0; k < kVec<ZB>; ++k)
    v[k] = __builtin_bit_cast(float, ZB ? (k & 1 ? r[k / 2] & 0xffff0000u : r[k / 2] << 16) : r[k]);
}

// Elements of a vector from its thread's element number `rest` on as -infinity.
template <bool ZB>
__device__ __forceinline__ void cut_vector(u32x4_t& r, int rest) {
  constexpr uint32_t kLow = ZB ? 0xff80ff80u : 0xff800000u;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if constexpr (ZB)
      r[k] = 2 * k >= rest ? kLow : 2 * k + 1 >= rest ? (r[k] & 0xffffu) | (kLow & 0xffff0000u) : r[k];
    else
      r[k] = k >= rest ? kLow : r[k];
  }
}

// A vector's elements into a maximum m and a sum s of 2^((v - m) c).
template <bool ZB>
__device__ __forceinline__ void running(const u32x4_t& r, float c, float& m, float& s) {
  float v[kVec<ZB>], most = m;
  unpack<ZB>(r, v);
#pragma unroll
  for (int k = 0; k < kVec<ZB>; ++k) most = fmaxf(most, v[k]);
  const float mf = finite_max(most);
  s *= exp2_fast((m - mf) * c);
#pragma unroll
  for (int k = 0; k < kVec<ZB>; ++k) s += exp2_fast((v[k] - mf) * c);
  m = most;
}

// A vector's gradients at byte offsets voff + soff of a row's window.
template <bool GB, int E>
__device__ __forceinline__ void store_gradient(__amdgpu_buffer_rsrc_t out, uint32_t voff, uint32_t soff,
                                               const float (&v)[E]) {
  const f32x4_t lo = {v[0], v[1], v[2], v[3]};
  if constexpr (E == 8) {
    const f32x4_t hi = {v[4], v[5], v[6], v[7]};
    if constexpr (GB) {
      const u32x2_t a = pack_bf16x4(lo), b = pack_bf16x4(hi);
      store16(out, voff, soff, u32x4_t{a[0], a[1], b[0], b[1]});
    } else {
      store16(out, voff, soff, lo);
      store16(out, voff + 16u, soff, hi);
    }
  } else {
    store4<GB ? 2 : 4>(out, voff, soff, lo);
  }
}

// The gradients of the row's entries with ids in [lo, hi), behind a barrier after
// the columns: the first entry of an id writes it, with the q of all of them.
// Up to 16 threads share an entry, each looking through its part of the others.
template <int THREADS, bool GB>
__device__ __forceinline__ void entry_gradients(const DistillArgs& a, int64_t row, const Entries& e, int lo,
                                                int hi, float coef, float m, float s, float total) {
  int share = 0;                                       // log2 of the threads of an entry
  while (share < 4 && (a.K << (share + 1)) <= THREADS) ++share;
  const int sub = threadIdx.x & ((1 << share) - 1);
  for (int j0 = 0; j0 < a.K; j0 += THREADS >> share) {
    const int j = j0 + (int(threadIdx.x) >> share);
    const int id = j < a.K ? e.id[j] : -1;
    const bool mine = id >= lo && id < hi;
    float q = 0.0f;
    uint32_t again = 0;
    if (mine)
      for (int k = 4 * sub; k < a.K; k += 4 << share) {
        const i32x4_t ids = *reinterpret_cast<const i32x4_t*>(&e.id[k]);
        const f32x4_t qs = *reinterpret_cast<const f32x4_t*>(&e.q[k]);
#pragma unroll
        for (int n = 0; n < 4; ++n)
          if (ids[n] == id) {
            again |= uint32_t(k + n < j);
            q += qs[n];
          }
      }
    // As row16_all, over the entry's threads.
    auto join = [&](auto ctrl) {
      q += lanes_dpp<decltype(ctrl)::value>(q);
      again |= lanes_dpp<decltype(ctrl)::value>(again);
    };
    if (share > 0) join(std::integral_constant<int, 0xB1>{});
    if (share > 1) join(std::integral_constant<int, 0x4E>{});
    if (share > 2) join(std::integral_constant<int, 0x141>{});
    if (share > 3) join(std::integral_constant<int, 0x140>{});
    if (mine && sub == 0 && !again) {
      const float g = coef * (exp2_fast((e.z[j] - m) * a.c) / s - q / total);
      if constexpr (GB)
        static_cast<__bf16*>(a.grad)[row * a.ld + id] = __bf16(g);
      else
        static_cast<float*>(a.grad)[row * a.ld + id] = g;
    }
  }
}

// An entry's share of tau times the loss, without the logarithms of the two sums.
__device__ __forceinline__ float entry_loss(const DistillArgs& a, float u, float top, float total, float z,
                                            float m) {
  const float du = u - top, q = exp2_fast(du * a.c) / total;
  return q != 0.0f ? q * (du - (z - m)) : 0.0f;
}

// A row's loss from its entries' shares l. Those count tau, the logarithms tau^2, which
// float32 may not hold where it holds tau (below 1e-19): then they do not count either.
__device__ __forceinline__ float row_loss(const DistillArgs& a, float w, float l, float s, float total) {
  return w * __builtin_fmaf(a.grad_scale, l, a.loss_scale * (logf(s) - logf(total)));
}

// --------------------------------------------------------------------------
// few rows: chunks
// --------------------------------------------------------------------------
constexpr int kChunkThreads = 256;
constexpr int kChunkColumns = 16 * kChunkThreads;

// Whether loads go out before it is known that the row counts (its weight is not 0): at
// most a workgroup to a CU, so that latency is all there is. More of them wait for the
// weight and read no row of weight 0.
__device__ __forceinline__ bool eager(const DistillArgs& a) { return a.items <= 256; }

// The chunk's vectors of a thread, zeros past the row's end.
template <bool ZB>
__device__ __forceinline__ void load_chunk(const DistillArgs& a, int64_t row, int first,
                                           u32x4_t (&raw)[16 / kVec<ZB>]) {
  constexpr int E = kVec<ZB>, S = ZB ? 2 : 4;
  const int columns = min((a.V + 7) / 8 * 8 - first, kChunkColumns);
  const __amdgpu_buffer_rsrc_t r =
      window(static_cast<const char*>(a.z) + (row * a.ld + first) * S, int64_t(columns) * S);
#pragma unroll
  for (int i = 0; i < 16 / E; ++i)
    raw[i] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
        r, int(threadIdx.x) * 16, i * kChunkThreads * 16, 0));
}

// Columns past V as -infinity.
template <bool ZB>
__device__ __forceinline__ void cut_chunk(const DistillArgs& a, int first, u32x4_t (&raw)[16 / kVec<ZB>]) {
  constexpr int E = kVec<ZB>;
  if (first + kChunkColumns > a.V)
#pragma unroll
    for (int i = 0; i < 16 / E; ++i)
      cut_vector<ZB>(raw[i], a.V - first - (i * kChunkThreads + int(threadIdx.x)) * E);
}

// What a thread loads of its entries, as it lies in memory: halves of the ids and of the
// teacher's logits, by the same instructions for either type. No load waits for another
// one, nor for the side of a branch that was not taken.
constexpr int kChunkEntries = kDistillMaxK / kChunkThreads;
struct EntryWords {
  uint32_t lo[kChunkEntries], hi[kChunkEntries], u0[kChunkEntries], u1[kChunkEntries];

  __device__ __forceinline__ void load_ids(const DistillArgs& a, int64_t row, bool look) {
    const int K = look ? a.K : 0, wide = a.wide_ids;
    const uint32_t* const p = static_cast<const uint32_t*>(a.ids) + (row * a.K << wide);
#pragma unroll
    for (int e = 0; e < kChunkEntries; ++e) {
      const int j = e * kChunkThreads + int(threadIdx.x);
      lo[e] = hi[e] = ~0u;
      if (j < K) {
        lo[e] = p[j << wide];
        hi[e] = p[(j << wide) + wide];               // the same word again where there is one
      }
    }
  }
  __device__ __forceinline__ void load_logits(const DistillArgs& a, int64_t row, bool look) {
    const int K = look ? a.K : 0, wide = !a.teacher_bf16;
    const uint16_t* const p = static_cast<const uint16_t*>(a.teacher) + (row * a.K << wide);
#pragma unroll
    for (int e = 0; e < kChunkEntries; ++e) {
      const int j = e * kChunkThreads + int(threadIdx.x);
      u0[e] = u1[e] = 0;
      if (j < K) {
        u0[e] = p[j << wide];
        u1[e] = p[(j << wide) + wide];
      }
    }
  }
  // The compiler may not look into the words before this point.
  __device__ __forceinline__ void arrived_ids() {
#pragma unroll
    for (int e = 0; e < kChunkEntries; ++e) asm volatile("" : "+v"(lo[e]), "+v"(hi[e]));
  }
  __device__ __forceinline__ void arrived_logits() {
#pragma unroll
    for (int e = 0; e < kChunkEntries; ++e) asm volatile("" : "+v"(u0[e]), "+v"(u1[e]));
  }
  // The column, -1 where there is none. V is below 2^31.
  __device__ __forceinline__ int id(const DistillArgs& a, int e) const {
    return (!a.wide_ids || hi[e] == 0) && lo[e] < uint32_t(a.V) ? int(lo[e]) : -1;
  }
  __device__ __forceinline__ float logit(const DistillArgs& a, int e) const {
    return __builtin_bit_cast(float, u1[e] << 16 | (a.teacher_bf16 ? 0u : u0[e]));
  }
};

template <bool ZB>
__global__ __launch_bounds__(kChunkThreads) void distill_stats_kernel(DistillArgs a) {
  constexpr int E = kVec<ZB>, W = kChunkThreads / 64;
  __shared__ float2 part[W];
  const int64_t item = blockIdx.x;
  const int64_t row = item / a.chunks;
  const int first = int(item - row * a.chunks) * kChunkColumns;
  if (!eager(a) && a.weight && a.weight[row] == 0.0f) return;
  EntryWords words;
  words.load_ids(a, row, true);
  u32x4_t raw[16 / E];
  load_chunk<ZB>(a, row, first, raw);
  words.arrived_ids();
  int id[kChunkEntries];                             // of entries in this chunk
  uint32_t zt[kChunkEntries];
#pragma unroll
  for (int e = 0; e < kChunkEntries; ++e) {
    id[e] = words.id(a, e);
    if (id[e] < first || id[e] >= first + kChunkColumns) id[e] = -1;
    zt[e] = 0;
    if (id[e] >= 0) {
      const int64_t at = row * a.ld + id[e];
      zt[e] = ZB ? static_cast<const uint16_t*>(a.z)[at] : static_cast<const uint32_t*>(a.z)[at];
    }
  }
  cut_chunk<ZB>(a, first, raw);
  float m = -INFINITY, s = 0.0f, v[E];
#pragma unroll
  for (int i = 0; i < 16 / E; ++i) {
    unpack<ZB>(raw[i], v);
#pragma unroll
    for (int k = 0; k < E; ++k) m = fmaxf(m, v[k]);
  }
  m = wave_max(m);
  const float mf = finite_max(m);
#pragma unroll
  for (int i = 0; i < 16 / E; ++i) {
    unpack<ZB>(raw[i], v);
#pragma unroll
    for (int k = 0; k < E; ++k) s += exp2_fast((v[k] - mf) * a.c);
  }
#pragma unroll
  for (int e = 0; e < kChunkEntries; ++e) {
    asm volatile("" : "+v"(zt[e]));                  // not looked into before
    if (id[e] >= 0)
      a.logit[row * a.K + e * kChunkThreads + int(threadIdx.x)] =
          __builtin_bit_cast(float, ZB ? zt[e] << 16 : zt[e]);
  }
  s = wave_sum(s);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = make_float2(m, s);
  __syncthreads();
  if (threadIdx.x == 0) {
    float most = part[0].x, sum = 0.0f;
#pragma unroll
    for (int w = 1; w < W; ++w) most = fmaxf(most, part[w].x);
#pragma unroll
    for (int w = 0; w < W; ++w)
      sum += part[w].y * exp2_fast((part[w].x - finite_max(most)) * a.c);
    a.stats[item] = make_float2(most, sum);
  }
}

template <bool ZB, bool GB>
__global__ __launch_bounds__(kChunkThreads) void distill_gradient_kernel(DistillArgs a) {
  constexpr int E = kVec<ZB>, N = kChunkThreads, W = N / 64, EPT = kChunkEntries, GS = GB ? 2 : 4;
  __shared__ __attribute__((aligned(16))) Entries entry;
  __shared__ float part[4][W];
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63;
  const int64_t item = blockIdx.x;
  const int64_t row = item / a.chunks_out;
  const int chunk = int(item - row * a.chunks_out), first = chunk * kChunkColumns;
  float w = 1.0f;
  if (!eager(a) && a.weight) w = a.weight[row];
  const bool look = eager(a) || w != 0.0f;
  u32x4_t raw[16 / E];
  if (look && a.grad) load_chunk<ZB>(a, row, first, raw);
  EntryWords words;
  words.load_ids(a, row, look);
  words.load_logits(a, row, look);
  int id[EPT];
  float u[EPT], zt[EPT], top = -INFINITY, total = 0.0f;
#pragma unroll
  for (int e = 0; e < EPT; ++e) {
    const int j = e * N + tid;
    zt[e] = j < a.K && look ? a.logit[row * a.K + j] : 0.0f;     // means nothing where there is no id
  }
  if (eager(a) && a.weight) w = a.weight[row];
  // The row's maximum and sum from its chunks', by each wave for itself.
  float m = -INFINITY, s = 0.0f;
  if (look) {
    for (int k = lane; k < a.chunks; k += 64) {
      const float2 st = a.stats[row * a.chunks + k];
      const float most = fmaxf(m, st.x), mf = finite_max(most);
      s = s * exp2_fast((m - mf) * a.c) + st.y * exp2_fast((st.x - mf) * a.c);
      m = most;
    }
    const float mine = m;
    m = finite_max(wave_max(m));
    s = wave_sum(s * exp2_fast((mine - m) * a.c));
  }
  // Entries: each wave's largest and sum, joined behind the barrier.
  words.arrived_ids();
  words.arrived_logits();
#pragma unroll
  for (int e = 0; e < EPT; ++e) {
    id[e] = w != 0.0f ? words.id(a, e) : -1;
    u[e] = words.logit(a, e);
    if (u[e] == -INFINITY) id[e] = -1;
    if (id[e] >= 0) top = fmaxf(top, u[e]);
  }
  bool some = false;
#pragma unroll
  for (int e = 0; e < EPT; ++e) some = some || id[e] >= 0;
  if (look && a.grad) cut_chunk<ZB>(a, first, raw);
  top = wave_max(top);
  const bool any = __ballot(some) != 0;
  if (lane == 0) {
    part[0][wave] = top;
    part[1][wave] = any ? 1.0f : 0.0f;
  }
  __syncthreads();
  top = -INFINITY;
  float live = 0.0f;
#pragma unroll
  for (int k = 0; k < W; ++k) {
    top = fmaxf(top, part[0][k]);
    live = fmaxf(live, part[1][k]);
  }
  top = finite_max(top);
#pragma unroll
  for (int e = 0; e < EPT; ++e) {
    const int j = e * N + tid;
    const float q = id[e] >= 0 ? exp2_fast((u[e] - top) * a.c) : 0.0f;
    total += q;
    if (j < (a.K + 3 & ~3)) {                        // up to a multiple of 4
      entry.id[j] = id[e];
      entry.q[j] = q;
      entry.z[j] = zt[e];
    }
  }
  total = wave_sum(total);
  if (lane == 0) part[2][wave] = total;
  __syncthreads();
  total = 0.0f;
#pragma unroll
  for (int k = 0; k < W; ++k) total += part[2][k];
  const float coef = a.grad_scale * w, inv = 1.0f / s;
  if (a.grad) {
    const int shown = live != 0.0f ? a.V - first : 0;            // columns of the chunk that count
    const int columns = int(min(a.ld - first, int64_t(kChunkColumns)));
    const __amdgpu_buffer_rsrc_t out =
        window(static_cast<char*>(a.grad) + (row * a.ld + first) * GS, int64_t(columns) * GS);
#pragma unroll
    for (int i = 0; i < 16 / E; ++i) {
      const int c = (i * N + tid) * E;
      float v[E] = {};
      if (c < shown) {
        unpack<ZB>(raw[i], v);
#pragma unroll
        for (int k = 0; k < E; ++k)
          v[k] = c + k < shown ? coef * (exp2_fast((v[k] - m) * a.c) * inv) : 0.0f;
      }
      store_gradient<GB, E>(out, uint32_t(tid * E * GS), uint32_t(i * N * E * GS), v);
    }
  }
  if (chunk == 0) {
    float l = 0.0f;
#pragma unroll
    for (int e = 0; e < EPT; ++e)
      if (id[e] >= 0) l += entry_loss(a, u[e], top, total, zt[e], m);
    l = wave_sum(l);
    if (lane == 0) part[3][wave] = l;
  }
  __syncthreads();
  if (chunk == 0 && tid == 0) {
    float l = 0.0f;
#pragma unroll
    for (int k = 0; k < W; ++k) l += part[3][k];
    a.loss[row] = live != 0.0f ? row_loss(a, w, l, s, total) : 0.0f;
  }
  if (a.grad && live != 0.0f)
    entry_gradients<N, GB>(a, row, entry, first, first + kChunkColumns, coef, m, s, total);
}

// --------------------------------------------------------------------------
// rows in registers
// --------------------------------------------------------------------------

// The compiler may not keep what it made of r before, and compares n anew where it
// is used (16 comparisons kept as masks fill the scalar registers).
__device__ __forceinline__ void forget(u32x4_t& r) { asm volatile("" : "+v"(r)); }
__device__ __forceinline__ int anew(int n) {
  asm volatile("" : "+s"(n));
  return n;
}

template <bool ZB, bool GB, int THREADS, int NV>
__global__ __launch_bounds__(THREADS) __attribute__((amdgpu_waves_per_eu(4)))
void distill_rows_kernel(DistillArgs a) {
  constexpr int E = kVec<ZB>, W = THREADS / 64, EPT = (kDistillMaxK + THREADS - 1) / THREADS;
  constexpr int kBlock = THREADS * E;                  // columns of one load instruction of all waves
  constexpr int ZS = ZB ? 2 : 4, GS = GB ? 2 : 4, kAhead = NV < 8 ? 2 : 3;
  __shared__ __attribute__((aligned(16))) Entries entry;
  __shared__ float part[6][W];
  const int tid = threadIdx.x, wave = tid >> 6;
  const uint32_t vz = uint32_t(tid * E * ZS);
  u32x4_t raw[NV];
  int id[EPT];
  float u[EPT], zt[EPT];

  // A row that is not looked at has an empty window: its loads cost no memory access.
  auto row_window = [&](int64_t row, bool wanted) {
    return window(static_cast<const char*>(a.z) + (wanted ? row * a.ld * ZS : 0),
                  wanted ? int64_t(a.V + 7) / 8 * 8 * ZS : 0);
  };
  // Block i of a row: zeros past its end.
  auto load = [&](__amdgpu_buffer_rsrc_t r, int i) {
    return __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, int(vz), i * kBlock * ZS, kStatePolicy));
  };
  // Blocks before `full` are whole, block `full` has `rest` columns or none.
  const int full = a.V / kBlock, rest = a.V - full * kBlock, blocks = full + (rest > 0);
  auto cut = [&](u32x4_t& r) { cut_vector<ZB>(r, rest - tid * E); };
  // The entries' numbers, then what belongs to those within the vocabulary.
  auto load_ids = [&](int64_t row, bool wanted, int64_t (&n)[EPT]) {
#pragma unroll
    for (int e = 0; e < EPT; ++e) {
      const int j = e * THREADS + tid;
      n[e] = -1;
      if (wanted && j < a.K) n[e] = entry_id(a, row * a.K + j);
    }
  };
  auto load_logits = [&](int64_t row, const int64_t (&n)[EPT]) {
#pragma unroll
    for (int e = 0; e < EPT; ++e) {
      const int j = e * THREADS + tid;
      id[e] = -1;
      u[e] = zt[e] = 0.0f;
      if (n[e] >= 0 && n[e] < a.V) {
        id[e] = int(n[e]);
        u[e] = entry_logit(a, row * a.K + j);
        zt[e] = student_logit<ZB>(a, row * a.ld + n[e]);
      }
    }
  };
  // op over the waves' numbers: 16 lanes have one each, so that few registers do.
  const int part_lane = tid & 15;
  auto of_wave = [&](const float* p, float none) { return part_lane < W ? p[part_lane] : none; };
  auto combine = [&](float v, auto op) { return row16_all(v, op); };
  auto add = [](float x, float y) { return x + y; };
  auto larger = [](float x, float y) { return fmaxf(x, y); };

  // Vector i, which is held, into the thread's maximum and sum, if its row has `shown`
  // blocks that count.
  float mine_m = -INFINITY, mine_s = 0.0f;
  auto take = [&](int i, int shown) {
    if (i == anew(full)) cut(raw[i]);
    if (i < anew(shown)) running<ZB>(raw[i], a.c, mine_m, mine_s);
    forget(raw[i]);
    __builtin_amdgcn_sched_barrier(0);
  };

  const int64_t step = gridDim.x;
  int64_t row = blockIdx.x;
  float w = row >= a.T ? 0.0f : a.weight ? a.weight[row] : 1.0f;
  {
    const __amdgpu_buffer_rsrc_t r = row_window(row, w != 0.0f);
#pragma unroll
    for (int i = 0; i < NV; ++i) raw[i] = load(r, i);
    int64_t n[EPT];
    load_ids(row, w != 0.0f, n);
    load_logits(row, n);
#pragma unroll
    for (int i = 0; i < NV; ++i) take(i, w != 0.0f ? blocks : 0);
  }
  for (; row < a.T; row += step) {
    const int64_t next = row + step;
    const float wn = next >= a.T ? 0.0f : a.weight ? a.weight[next] : 1.0f;
    const bool ahead = wn != 0.0f;                     // the next row is loaded meanwhile
    const __amdgpu_buffer_rsrc_t here = row_window(row, w != 0.0f), there = row_window(next, ahead);
    int64_t ids[EPT];
    load_ids(next, ahead, ids);
    // Block i of a row that is longer than what is held.
    auto streamed = [&](int i) {
      u32x4_t r = load(here, i);
      if (i == full) cut(r);
      return r;
    };
    // The blocks that are not held.
    for (int i = NV; i < (w != 0.0f ? blocks : 0); ++i) running<ZB>(streamed(i), a.c, mine_m, mine_s);
    float top = -INFINITY;
    bool some = false;
#pragma unroll
    for (int e = 0; e < EPT; ++e) {
      if (u[e] == -INFINITY) id[e] = -1;
      if (id[e] >= 0) {
        top = fmaxf(top, u[e]);
        some = true;
      }
    }
    float m = wave_max(mine_m);
    float s = wave_sum(mine_s * exp2_fast((mine_m - finite_max(m)) * a.c));
    top = wave_max(top);
    const bool any = __ballot(some) != 0;
    if ((tid & 63) == 0) {
      part[0][wave] = m;
      part[1][wave] = top;
      part[2][wave] = any ? 1.0f : 0.0f;
      part[3][wave] = s;
    }
    __syncthreads();
    const float wave_m = of_wave(part[0], -INFINITY);
    m = finite_max(combine(wave_m, larger));
    s = combine(of_wave(part[3], 0.0f) * exp2_fast((wave_m - m) * a.c), add);
    top = finite_max(combine(of_wave(part[1], -INFINITY), larger));
    const bool live = __builtin_amdgcn_readfirstlane(int(combine(of_wave(part[2], 0.0f), larger))) != 0;
    const int shown = live ? blocks : 0;

    float total = 0.0f;
    if (live)
#pragma unroll
      for (int e = 0; e < EPT; ++e) {
        const int j = e * THREADS + tid;
        const float q = id[e] >= 0 ? exp2_fast((u[e] - top) * a.c) : 0.0f;
        total += q;
        if (j < (a.K + 3 & ~3)) {              // up to a multiple of 4
          entry.id[j] = id[e];
          entry.q[j] = q;
          entry.z[j] = zt[e];
        }
      }
    total = wave_sum(total);
    if ((tid & 63) == 0) part[4][wave] = total;
    __syncthreads();
    total = combine(of_wave(part[4], 0.0f), add);
    if (live) {
      float l = 0.0f;
#pragma unroll
      for (int e = 0; e < EPT; ++e)
        if (id[e] >= 0) l += entry_loss(a, u[e], top, total, zt[e], m);
      l = wave_sum(l);
      if ((tid & 63) == 0) part[5][wave] = l;
    }
    load_logits(next, ids);                            // this row's are in LDS
    const float coef = a.grad_scale * w;
    const float inv = 1.0f / s;
    const __amdgpu_buffer_rsrc_t out =
        window(static_cast<char*>(a.grad) + row * a.ld * GS, a.ld * GS);
    auto emit = [&](const u32x4_t& r, int i) {
      float v[E] = {};
      if (i < anew(shown)) {
        unpack<ZB>(r, v);
#pragma unroll
        for (int k = 0; k < E; ++k) v[k] = coef * (exp2_fast((v[k] - m) * a.c) * inv);
      }
      store_gradient<GB, E>(out, uint32_t(tid * E * GS), uint32_t(i * kBlock * GS), v);
    };
    const int out_blocks = int((a.ld + kBlock - 1) / kBlock);
    // As vectors leave, the next row's come, and are added up kAhead of them later: with
    // the sums behind the last store the memory waits for them (4096 x 128256 431 us, so
    // 411). 3, 6 or 10 vectors: 1021 x 32003 42.4, 43.4, 44.6 us, the others within 1%.
    mine_m = -INFINITY;
    mine_s = 0.0f;
    const int coming = ahead ? blocks : 0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (i < anew(out_blocks)) emit(raw[i], i);
      raw[i] = load(there, i);
      __builtin_amdgcn_sched_barrier(0);
      if (i >= kAhead) take(i - kAhead, coming);
    }
    for (int i = NV; i < out_blocks; ++i) emit(streamed(i), i);
    __syncthreads();
    const float l = combine(of_wave(part[5], 0.0f), add);
    if (tid == 0)
      a.loss[row] = live ? row_loss(a, w, l, s, total) : 0.0f;
    if (live) {
      entry_gradients<THREADS, GB>(a, row, entry, 0, a.V, coef, m, s, total);
      // Columns past V of the last block that counts: 0 times a sum that is not finite is not 0.
      const int64_t end = min(a.ld, int64_t(blocks) * kBlock);
      for (int64_t c = a.V + tid; c < end; c += THREADS) {
        if constexpr (GB)
          static_cast<uint16_t*>(a.grad)[row * a.ld + c] = 0;
        else
          static_cast<float*>(a.grad)[row * a.ld + c] = 0.0f;
      }
    }
#pragma unroll
    for (int i = NV - kAhead; i < NV; ++i) take(i, coming);
    w = wn;
  }
}

// --------------------------------------------------------------------------
// the loss alone
// --------------------------------------------------------------------------
//
// One pass over a row, each thread with a running maximum and a sum that is scaled
// when the maximum moves, kVec elements at a time: nothing is held, so several
// workgroups share a CU. Four loads are ahead of the four being added.
constexpr int kLossThreads = 512;
template <bool ZB>
__global__ __launch_bounds__(kLossThreads) void distill_loss_kernel(DistillArgs a) {
  constexpr int E = kVec<ZB>, W = kLossThreads / 64, EPT = kDistillMaxK / kLossThreads, U = 4;
  constexpr int kBlock = kLossThreads * E, ZS = ZB ? 2 : 4;
  __shared__ float part[6][W];
  const int tid = threadIdx.x, wave = tid >> 6;
  const int full = a.V / kBlock, rest = a.V - full * kBlock, blocks = full + (rest > 0);
  for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x) {
    const float w = a.weight ? a.weight[row] : 1.0f;
    if (w == 0.0f) {
      if (tid == 0) a.loss[row] = 0.0f;
      continue;
    }
    const __amdgpu_buffer_rsrc_t r =
        window(static_cast<const char*>(a.z) + row * a.ld * ZS, int64_t(a.V + 7) / 8 * 8 * ZS);
    u32x4_t raw[2][U];
    auto load = [&](u32x4_t (&to)[U], int i) {         // past the row's end: zeros, not looked at
#pragma unroll
      for (int k = 0; k < U; ++k)
        to[k] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
            r, tid * 16, (i + k) * kLossThreads * 16, kStatePolicy));
    };
    load(raw[0], 0);
    int id[EPT];
    float u[EPT], zt[EPT], top = -INFINITY;
    bool some = false;
#pragma unroll
    for (int e = 0; e < EPT; ++e) {
      const int j = e * kLossThreads + tid;
      id[e] = -1;
      u[e] = zt[e] = 0.0f;
      if (j < a.K) {
        const int64_t n = entry_id(a, row * a.K + j);
        if (n >= 0 && n < a.V) {
          u[e] = entry_logit(a, row * a.K + j);
          zt[e] = student_logit<ZB>(a, row * a.ld + n);
          if (u[e] != -INFINITY) {
            id[e] = int(n);
            top = fmaxf(top, u[e]);
            some = true;
          }
        }
      }
    }
    float m = -INFINITY, s = 0.0f;
    auto add = [&](u32x4_t v4, int i) {
      if (i >= blocks) return;
      if (i == full) cut_vector<ZB>(v4, rest - tid * E);
      running<ZB>(v4, a.c, m, s);
    };
    for (int i = 0; i < blocks; i += 2 * U) {
      load(raw[1], i + U);
#pragma unroll
      for (int k = 0; k < U; ++k) add(raw[0][k], i + k);
      load(raw[0], i + 2 * U);
#pragma unroll
      for (int k = 0; k < U; ++k) add(raw[1][k], i + U + k);
    }
    // The waves' maxima and sums, then all of them.
    const float mine = m;
    m = wave_max(m);
    s = wave_sum(s * exp2_fast((mine - finite_max(m)) * a.c));
    top = wave_max(top);
    const bool any = __ballot(some) != 0;
    if ((tid & 63) == 0) {
      part[0][wave] = m;
      part[1][wave] = s;
      part[2][wave] = top;
      part[3][wave] = any ? 1.0f : 0.0f;
    }
    __syncthreads();
    float live = 0.0f;
#pragma unroll
    for (int k = 0; k < W; ++k) {
      m = fmaxf(m, part[0][k]);
      top = fmaxf(top, part[2][k]);
      live = fmaxf(live, part[3][k]);
    }
    m = finite_max(m);
    top = finite_max(top);
    s = 0.0f;
#pragma unroll
    for (int k = 0; k < W; ++k) s += part[1][k] * exp2_fast((part[0][k] - m) * a.c);
    float total = 0.0f;
#pragma unroll
    for (int e = 0; e < EPT; ++e)
      if (id[e] >= 0) total += exp2_fast((u[e] - top) * a.c);
    total = wave_sum(total);
    if ((tid & 63) == 0) part[4][wave] = total;
    __syncthreads();
    total = 0.0f;
#pragma unroll
    for (int k = 0; k < W; ++k) total += part[4][k];
    float l = 0.0f;
#pragma unroll
    for (int e = 0; e < EPT; ++e)
      if (id[e] >= 0) l += entry_loss(a, u[e], top, total, zt[e], m);
    l = wave_sum(l);
    if ((tid & 63) == 0) part[5][wave] = l;
    __syncthreads();
    if (tid == 0) {
      l = 0.0f;
#pragma unroll
      for (int k = 0; k < W; ++k) l += part[5][k];
      a.loss[row] = live != 0.0f ? row_loss(a, w, l, s, total) : 0.0f;
    }
  }
}

}  // namespace forge
