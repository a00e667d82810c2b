// Distillation from a teacher's top logits for gfx950: each row's loss and the
// gradient of the student's logits.
//
//   q = softmax(u / tau) over the row's entries, p = softmax(z / tau) over V columns
//   loss = scale w tau^2 sum_j q_j (log q_j - log p[id_j])
//   dz_i = scale w tau (p_i - sum of the q_j with id_j == i)
//
// Bound by HBM: the logits are read and the gradient is written. A row is cut into
// chunks, a workgroup each: the first launch forms each chunk's maximum and sum
// of exponentials, the second joins a row's chunks and forms the gradient. The
// teacher's columns are written with the others and once more, with their q,
// behind a barrier: the workgroup that has the column does both.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

#include "row_io.hpp"

namespace forge {

constexpr int kDistillThreads = 256;
constexpr int kDistillMaxK = 1024;

struct DistillArgs {
  const void *z, *teacher, *ids;
  const float* weight;               // NULL: 1
  float* loss;
  void* grad;                        // NULL: the loss alone
  float2* stats;                     // [T][chunks]: maximum, sum of 2^((z - maximum) c)
  float* logit;                      // [T][K]: the student's logit of each entry
  int64_t T, ld, items;              // items: rows times chunks of the launch
  int32_t V, K, chunks, chunks_out;  // chunks of V and of ld columns
  int32_t wide_ids, teacher_bf16;
  float c, inv_tau, loss_scale, grad_scale;    // log2(e) / tau, 1 / tau, scale tau^2, scale tau
};

// The row's entries in LDS: ids (-1: not there) and q, as they are formed.
struct Entries {
  int32_t id[kDistillMaxK];
  float q[kDistillMaxK];
};

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// Maximum and sum over the workgroup, in every thread. `part`: a float for each wave.
template <int THREADS>
__device__ __forceinline__ float block_max(float v, float* part) {
  v = wave_max(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  v = part[0];
#pragma unroll
  for (int w = 1; w < THREADS / 64; ++w) v = fmaxf(v, part[w]);
  return v;
}
template <int THREADS>
__device__ __forceinline__ float block_total(float v, float* part) {
  v = wave_sum(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  v = part[0];
#pragma unroll
  for (int w = 1; w < THREADS / 64; ++w) v += part[w];
  return v;
}

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
// -infinity, so that a difference is -infinity and no NaN.
__device__ __forceinline__ float finite_max(float m) { return m == -INFINITY ? 0.0f : m; }

// Columns [first, first + 32 * THREADS) of a row to a thread's 32 registers: thread t
// has vectors t, t + THREADS and so on. Columns past V are -infinity.
template <bool ZB, int THREADS, int E>
__device__ __forceinline__ void load_chunk(const DistillArgs& a, int64_t row, int first,
                                           float (&v)[32 / E][E]) {
#pragma unroll
  for (int i = 0; i < 32 / E; ++i) {
    const int c = first + (i * THREADS + int(threadIdx.x)) * E;
    if (c < a.V) load_elems<ZB, E>(a.z, row * a.ld + c, v[i]);
#pragma unroll
    for (int k = 0; k < E; ++k)
      if (c + k >= a.V) v[i][k] = -INFINITY;
  }
}

template <bool ZB>
__global__ __launch_bounds__(kDistillThreads) void distill_stats_kernel(DistillArgs a) {
  constexpr int N = kDistillThreads, E = ZB ? 8 : 4;
  __shared__ float part[N / 64];
  for (int64_t item = blockIdx.x; item < a.items; item += gridDim.x) {
    const int64_t row = item / a.chunks;
    const int chunk = int(item - row * a.chunks);
    if (a.weight && a.weight[row] == 0.0f) continue;
    const int first = chunk * 32 * N;
    float v[32 / E][E];
    load_chunk<ZB, N, E>(a, row, first, v);
    for (int j = threadIdx.x; j < a.K; j += N) {
      const int64_t id = entry_id(a, row * a.K + j);
      if (id >= first && id < first + 32 * N && id < a.V)
        a.logit[row * a.K + j] = student_logit<ZB>(a, row * a.ld + id);
    }
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < 32 / E; ++i)
#pragma unroll
      for (int k = 0; k < E; ++k) m = fmaxf(m, v[i][k]);
    m = block_max<N>(m, part);
    const float ms = finite_max(m);
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 32 / E; ++i)
#pragma unroll
      for (int k = 0; k < E; ++k) s += exp2_fast((v[i][k] - ms) * a.c);
    s = block_total<N>(s, part);
    if (threadIdx.x == 0) a.stats[item] = make_float2(m, s);
  }
}

// The row's entries to LDS. False if there are none.
template <int THREADS>
__device__ __forceinline__ bool load_entries(const DistillArgs& a, int64_t row, Entries& e, float* part,
                                             float& top, float& sum) {
  float m = -INFINITY;
  bool some = false;
  __syncthreads();
  for (int j = threadIdx.x; j < a.K; j += THREADS) {
    const int64_t id = entry_id(a, row * a.K + j);
    bool kept = id >= 0 && id < a.V;
    const float u = kept ? entry_logit(a, row * a.K + j) : 0.0f;
    kept = kept && u != -INFINITY;
    e.id[j] = kept ? int32_t(id) : -1;
    e.q[j] = u;
    if (kept) m = fmaxf(m, u);
    some = some || kept;
  }
  if (!__syncthreads_or(some)) return false;
  m = finite_max(block_max<THREADS>(m, part));
  float s = 0.0f;
  for (int j = threadIdx.x; j < a.K; j += THREADS)
    if (e.id[j] >= 0) s += exp2_fast((e.q[j] - m) * a.c);
  top = m;
  sum = block_total<THREADS>(s, part);
  return true;
}

template <bool ZB, bool GB>
__global__ __launch_bounds__(kDistillThreads) void distill_gradient_kernel(DistillArgs a) {
  constexpr int N = kDistillThreads, E = io_elems<ZB, GB>;
  __shared__ float part[N / 64];
  __shared__ Entries entry;
  for (int64_t item = blockIdx.x; item < a.items; item += gridDim.x) {
    const int64_t row = item / a.chunks_out;
    const int chunk = int(item - row * a.chunks_out);
    const int first = chunk * 32 * N;
    const float w = a.weight ? a.weight[row] : 1.0f;
    float top, total;
    if (w == 0.0f || !load_entries<N>(a, row, entry, part, top, total)) {
      if (chunk == 0 && threadIdx.x == 0) a.loss[row] = 0.0f;
      if (a.grad) {
        const float zero[E] = {};
#pragma unroll
        for (int i = 0; i < 32 / E; ++i) {
          const int c = first + (i * N + int(threadIdx.x)) * E;
          if (c < a.ld) store_elems<GB, E>(a.grad, row * a.ld + c, zero);
        }
      }
      continue;
    }
    // The row's maximum and sum from its chunks'.
    float m = -INFINITY, s = 0.0f;
    for (int k = threadIdx.x; k < a.chunks; k += N) m = fmaxf(m, a.stats[row * a.chunks + k].x);
    m = finite_max(block_max<N>(m, part));
    for (int k = threadIdx.x; k < a.chunks; k += N) {
      const float2 st = a.stats[row * a.chunks + k];
      s += st.y * exp2_fast((finite_max(st.x) - m) * a.c);
    }
    s = block_total<N>(s, part);
    if (chunk == 0) {
      float l = 0.0f;
      for (int j = threadIdx.x; j < a.K; j += N)
        if (entry.id[j] >= 0) {
          const float du = entry.q[j] - top, q = exp2_fast(du * a.c) / total;
          if (q != 0.0f) l += q * (du * a.inv_tau - (a.logit[row * a.K + j] - m) * a.inv_tau);
        }
      l = block_total<N>(l, part);
      if (threadIdx.x == 0) a.loss[row] = a.loss_scale * w * (l + (logf(s) - logf(total)));
    }
    if (!a.grad) continue;
    const float inv = 1.0f / s, coef = a.grad_scale * w;
    float v[32 / E][E];
    load_chunk<ZB, N, E>(a, row, first, v);
#pragma unroll
    for (int i = 0; i < 32 / E; ++i) {
      const int c = first + (i * N + int(threadIdx.x)) * E;
#pragma unroll
      for (int k = 0; k < E; ++k)
        v[i][k] = c + k < a.V ? coef * (exp2_fast((v[i][k] - m) * a.c) * inv) : 0.0f;
      if (c < a.ld) store_elems<GB, E>(a.grad, row * a.ld + c, v[i]);
    }
    __syncthreads();
    // The teacher's columns: the first entry of an id writes it.
    for (int j = threadIdx.x; j < a.K; j += N) {
      const int id = entry.id[j];
      if (id < first || id >= first + 32 * N) continue;
      float q = 0.0f;
      bool again = false;
      for (int k = 0; k < a.K; ++k)
        if (entry.id[k] == id) {
          again = again || k < j;
          q += exp2_fast((entry.q[k] - top) * a.c);
        }
      if (again) continue;
      const float p = exp2_fast((a.logit[row * a.K + j] - m) * a.c) * inv;
      const float g[1] = {coef * (p - q / total)};
      if constexpr (GB)
        static_cast<__bf16*>(a.grad)[row * a.ld + id] = __bf16(g[0]);
      else
        static_cast<float*>(a.grad)[row * a.ld + id] = g[0];
    }
  }
}

}  // namespace forge
