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

typedef int i32x4_t __attribute__((ext_vector_type(4)));

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


// --------------------------------------------------------------------------
// rows in registers
// --------------------------------------------------------------------------

// A vector of 16 bytes of a row and its elements.
template <bool ZB>
constexpr int kVec = ZB ? 8 : 4;
template <bool ZB>
__device__ __forceinline__ void unpack(const u32x4_t& r, float (&v)[kVec<ZB>]) {
#pragma unroll
  for (int k = 0; k < kVec<ZB>; ++k)
    v[k] = __builtin_bit_cast(float, ZB ? (k & 1 ? r[k / 2] & 0xffff0000u : r[k / 2] << 16) : r[k]);
}

// The compiler may not keep what it made of r before.
__device__ __forceinline__ void forget(u32x4_t& r) { asm volatile("" : "+v"(r)); }

template <bool ZB, bool GB, bool GRAD, int THREADS, int NV>
__global__ __launch_bounds__(THREADS) void distill_rows_kernel(DistillArgs a) {
  constexpr int E = kVec<ZB>, W = THREADS / 64, EPT = (kDistillMaxK + THREADS - 1) / THREADS;
  constexpr int kBlock = THREADS * E;                  // columns of one load instruction of all waves
  constexpr int ZS = ZB ? 2 : 4, GS = GB ? 2 : 4;
  constexpr uint32_t kLow = ZB ? 0xff80ff80u : 0xff800000u;    // -infinity
  __shared__ __attribute__((aligned(16))) Entries entry;
  __shared__ float part[6][W];
  const int tid = threadIdx.x, wave = tid >> 6;
  const uint32_t vz = uint32_t(tid * E * ZS), vg = uint32_t(tid * E * GS);
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
  // Its elements past V as -infinity.
  auto cut = [&](u32x4_t& r) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (ZB) {
        const bool lo = tid * E + 2 * k >= rest, hi = tid * E + 2 * k + 1 >= rest;
        r[k] = lo ? kLow : hi ? (r[k] & 0xffffu) | (kLow & 0xffff0000u) : r[k];
      } else {
        r[k] = tid * E + k >= rest ? kLow : r[k];
      }
    }
  };
  auto load_entries_of = [&](int64_t row, int (&id)[EPT], float (&u)[EPT], float (&zt)[EPT]) {
#pragma unroll
    for (int e = 0; e < EPT; ++e) {
      const int j = e * THREADS + tid;
      id[e] = -1;
      u[e] = zt[e] = 0.0f;
      if (j < a.K) {
        const int64_t n = entry_id(a, row * a.K + j);
        if (n >= 0 && n < a.V) {
          u[e] = entry_logit(a, row * a.K + j);
          zt[e] = student_logit<ZB>(a, row * a.ld + n);
          if (u[e] != -INFINITY) id[e] = int(n);
        }
      }
    }
  };
  auto combine = [&](const float* p, auto op) {
    float v = p[0];
#pragma unroll
    for (int w = 1; w < W; ++w) v = op(v, p[w]);
    return v;
  };
  auto add = [](float x, float y) { return x + y; };
  auto larger = [](float x, float y) { return fmaxf(x, y); };

  const int64_t step = gridDim.x;
  int64_t row = blockIdx.x;
  float w = row >= a.T ? 0.0f : a.weight ? a.weight[row] : 1.0f;
  {
    const __amdgpu_buffer_rsrc_t r = row_window(row, w != 0.0f);
#pragma unroll
    for (int i = 0; i < NV; ++i) raw[i] = load(r, i);
    if (w != 0.0f) load_entries_of(row, id, u, zt);
  }
  for (; row < a.T; row += step) {
    const int64_t next = row + step;
    const float wn = next >= a.T ? 0.0f : a.weight ? a.weight[next] : 1.0f;
    const bool ahead = wn != 0.0f;                     // the next row is loaded meanwhile
    const __amdgpu_buffer_rsrc_t here = row_window(row, w != 0.0f), there = row_window(next, ahead);
    // Block i of a row that is longer than what is held.
    auto streamed = [&](int i) {
      u32x4_t r = load(here, i);
      if (i == full) cut(r);
      return r;
    };
    float m = -INFINITY, top = -INFINITY;
    bool some = false;
    auto most = [&](const u32x4_t& r) {
      float v[E];
      unpack<ZB>(r, v);
#pragma unroll
      for (int k = 0; k < E; ++k) m = fmaxf(m, v[k]);
    };
    int shown = w != 0.0f ? blocks : 0;                // blocks of the row that count
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (i == full) cut(raw[i]);
      if (i < shown) most(raw[i]);
      forget(raw[i]);
      __builtin_amdgcn_sched_barrier(0);
    }
    for (int i = NV; i < shown; ++i) most(streamed(i));
    if (w != 0.0f)
#pragma unroll
      for (int e = 0; e < EPT; ++e)
        if (id[e] >= 0) {
          top = fmaxf(top, u[e]);
          some = true;
        }
    m = wave_max(m);
    top = wave_max(top);
    const bool any = __ballot(some) != 0;
    if ((tid & 63) == 0) {
      part[0][wave] = m;
      part[1][wave] = top;
      part[2][wave] = any ? 1.0f : 0.0f;
    }
    __syncthreads();
    m = finite_max(combine(part[0], larger));
    top = finite_max(combine(part[1], larger));
    const bool live = combine(part[2], larger) != 0.0f;
    shown = live ? blocks : 0;

    float s = 0.0f, total = 0.0f;
    auto sum = [&](const u32x4_t& r) {
      float v[E];
      unpack<ZB>(r, v);
#pragma unroll
      for (int k = 0; k < E; ++k) s += exp2_fast((v[k] - m) * a.c);
    };
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (i < shown) sum(raw[i]);
      forget(raw[i]);
      if (!GRAD) raw[i] = load(there, i);
      __builtin_amdgcn_sched_barrier(0);
    }
    for (int i = NV; i < shown; ++i) sum(streamed(i));
    if (live)
#pragma unroll
      for (int e = 0; e < EPT; ++e) {
        const int j = e * THREADS + tid;
        const float q = id[e] >= 0 ? exp2_fast((u[e] - top) * a.c) : 0.0f;
        total += q;
        if (GRAD && j < (a.K + 3 & ~3)) {              // up to a multiple of 4
          entry.id[j] = id[e];
          entry.q[j] = q;
        }
      }
    s = wave_sum(s);
    total = wave_sum(total);
    if ((tid & 63) == 0) {
      part[3][wave] = s;
      part[4][wave] = total;
    }
    __syncthreads();
    s = combine(part[3], add);
    total = combine(part[4], add);
    if (live) {
      float l = 0.0f;
#pragma unroll
      for (int e = 0; e < EPT; ++e)
        if (id[e] >= 0) {
          const float du = u[e] - top, q = exp2_fast(du * a.c) / total;
          if (q != 0.0f) l += q * (du * a.inv_tau - (zt[e] - m) * a.inv_tau);
        }
      l = wave_sum(l);
      if ((tid & 63) == 0) part[5][wave] = l;
    }
    int nid[EPT];
    float nu[EPT], nz[EPT];
    if (ahead) load_entries_of(next, nid, nu, nz);
    if constexpr (GRAD) {
      const float coef = a.grad_scale * w, inv = 1.0f / s;
      const __amdgpu_buffer_rsrc_t out =
          window(static_cast<char*>(a.grad) + row * a.ld * GS, a.ld * GS);
      auto emit = [&](const u32x4_t& r, int i) {
        float v[E] = {};
        if (i < shown) {
          unpack<ZB>(r, v);
#pragma unroll
          for (int k = 0; k < E; ++k) v[k] = coef * (exp2_fast((v[k] - m) * a.c) * inv);
          if (i == full)                               // zeros past V, whatever the sums are
#pragma unroll
            for (int k = 0; k < E; ++k) v[k] = tid * E + k >= rest ? 0.0f : v[k];
        }
        const uint32_t at = uint32_t(i * kBlock * GS);
#pragma unroll
        for (int k = 0; k < E; k += 4) {
          const f32x4_t g = {v[k], v[k + 1], v[k + 2], v[k + 3]};
          if constexpr (GB && E == 8) {
            if (k == 0) {
              const u32x2_t lo = pack_bf16x4(g), hi = pack_bf16x4(f32x4_t{v[4], v[5], v[6], v[7]});
              store16(out, vg, at, u32x4_t{lo[0], lo[1], hi[0], hi[1]});
            }
          } else {
            store4<GS>(out, vg + k * GS, at, g);
          }
        }
      };
      const int out_blocks = int((a.ld + kBlock - 1) / kBlock);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (i < out_blocks) emit(raw[i], i);
        raw[i] = load(there, i);
        __builtin_amdgcn_sched_barrier(0);
      }
      for (int i = NV; i < out_blocks; ++i) emit(streamed(i), i);
    }
    __syncthreads();
    if (tid == 0)
      a.loss[row] = live ? a.loss_scale * w * (combine(part[5], add) + (logf(s) - logf(total))) : 0.0f;
    if constexpr (GRAD) {
      // The teacher's columns: the first entry of an id writes it.
      if (live)
#pragma unroll
        for (int e = 0; e < EPT; ++e)
          if (id[e] >= 0) {
            const int j = e * THREADS + tid;
            float q = 0.0f;
            bool again = false;
            for (int k = 0; k < a.K; k += 4) {
              const i32x4_t ids = *reinterpret_cast<const i32x4_t*>(&entry.id[k]);
              const f32x4_t qs = *reinterpret_cast<const f32x4_t*>(&entry.q[k]);
#pragma unroll
              for (int n = 0; n < 4; ++n)
                if (ids[n] == id[e]) {
                  again = again || k + n < j;
                  q += qs[n];
                }
            }
            if (!again) {
              const float g = a.grad_scale * w * (exp2_fast((zt[e] - m) * a.c) / s - q / total);
              if constexpr (GB)
                static_cast<__bf16*>(a.grad)[row * a.ld + id[e]] = __bf16(g);
              else
                static_cast<float*>(a.grad)[row * a.ld + id[e]] = g;
            }
          }
    }
    w = wn;
#pragma unroll
    for (int e = 0; e < EPT; ++e) {
      id[e] = nid[e];
      u[e] = nu[e];
      zt[e] = nz[e];
    }
  }
}

}  // namespace forge
