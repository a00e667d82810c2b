// Global gradient norm over a list of tensors, and the passes that use it:
// the clipped gradient and the clipped optimizer steps.
//
//   norm = sqrt(sum g^2),  coef = min(1, max_norm / (norm + 1e-6)),
//   step on coef * g, formed in registers.
//
// A list goes to a kernel as a table in its arguments (a captured graph then
// holds its own copy, and nothing is copied to the device). Tensors are cut
// into chunks; a workgroup finds the tensor of its chunk with one load of the
// table's chunk offsets and a ballot. Every tensor starts at a chunk of its
// own, so all vector accesses are aligned and only a tensor's last chunk is
// partial.
//
// Both passes are bound by HBM. The norm reads the gradient once; squares are
// formed and added in float64 (a float32 square is exact there, so neither
// overflow nor vanishing squares need a scaling pass), whose vector rate on
// CDNA4 is several times what the stream needs. The partial sums of a fixed
// assignment of chunks to workgroups are joined by one workgroup in a fixed
// order: no atomics, the same bits in every run.
#pragma once

#include <hip/hip_runtime.h>

#include "wgrad_kernels.hpp"

namespace forge {

// Tensors in one launch: the tables stay under 4 KB of kernel arguments.
constexpr int kNormTensors = 320;
constexpr int kClipTensors = 160;    // three addresses a tensor
constexpr int kAdamTensors = 128;    // four
constexpr int kChunk = 4096;         // elements of a chunk
constexpr int kNormGrid = 2048;      // most workgroups (and partial sums) of a norm launch
constexpr int kNormAlone = 24;       // chunks that one workgroup sums by itself

// N 16-bit numbers, two to a word, so that they come by scalar loads.
template <int N>
struct Halves {
  static_assert(N % 2 == 0, "two to a word");
  uint32_t w[N / 2];
  __host__ __device__ uint32_t operator[](int k) const { return w[k >> 1] >> (16 * (k & 1)) & 0xffffu; }
  void set(int k, uint32_t v) {
    const int s = 16 * (k & 1);
    w[k >> 1] = (w[k >> 1] & ~(0xffffu << s)) | v << s;
  }
};

// The tensors of one launch, A addresses each (of 16-byte aligned arrays below
// 2^52: 6 bytes). Tensor t has the chunks first[t] .. first[t + 1] - 1, the last
// of them with tail[t] & 8191 elements; bit 15 of tail[t] marks a bf16 gradient.
// A list of 300 tensors takes one launch for the norm and two for an
// SGD-momentum step; with 8-byte addresses it took two and three, and 24M
// elements 100 us instead of 94 (and one tensor's norm and clip 201 instead of 203).
template <int N_, int A_>
struct TensorTable {
  static constexpr int N = N_, A = A_;
  uint32_t low[A][N];
  Halves<N> high[A];
  int32_t first[N + 1];              // INT32_MAX past the last tensor's end
  Halves<N> tail;
  int32_t chunks;
  __device__ __forceinline__ void* p(int a, int t) const {
    // By way of the global address space, so that its accesses are global ones.
    typedef __attribute__((address_space(1))) void global_void;
    return (void*)(global_void*)((uint64_t(high[a][t]) << 32 | low[a][t]) << 4);
  }
  void set(int a, int t, const void* at, int64_t bytes) {
    const uint64_t u = (reinterpret_cast<uintptr_t>(at) + uint64_t(bytes)) >> 4;
    low[a][t] = uint32_t(u);
    high[a].set(t, uint32_t(u >> 32));
  }
};
typedef TensorTable<kNormTensors, 1> NormTable;     // gradient
typedef TensorTable<kClipTensors, 3> ClipTable;     // gradient, and its place or W and momentum
typedef TensorTable<kAdamTensors, 4> AdamTable;     // gradient, W, m, v
static_assert(sizeof(NormTable) <= 4000 && sizeof(ClipTable) <= 4000 && sizeof(AdamTable) <= 4000,
              "kernel argument size");

// The tensor of chunk c: the last one that starts at or before it. Every lane
// of the wave takes part.
template <class Table>
__device__ __forceinline__ int tensor_of(const Table& tab, int c) {
  constexpr int N = Table::N;
  const int lane = threadIdx.x & 63;
  int t = -1;
#pragma unroll
  for (int k = 0; k < N; k += 64) {
    const bool below = k + lane < N && tab.first[k + lane < N ? k + lane : N - 1] <= c;
    t += __popcll(__ballot(below));
  }
  return __builtin_amdgcn_readfirstlane(t);
}

// Elements of tensor t that lie before the end of its chunk c.
template <class Table>
__device__ __forceinline__ int64_t end_of(const Table& tab, int t, int c) {
  const int64_t k = int64_t(c - tab.first[t]) * kChunk;
  return k + (c + 1 == tab.first[t + 1] || c + 1 == tab.chunks ? tab.tail[t] & 8191 : kChunk);
}

// Sum of v over the workgroup, in thread 0. `part`: one double per wave.
__device__ __forceinline__ double block_sum(double v, double* part) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_down(v, d);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
  __syncthreads();
  if (threadIdx.x == 0) {
    v = 0.0;
    for (int w = 0; w < int(blockDim.x >> 6); ++w) v += part[w];
  }
  return v;
}

__device__ __forceinline__ void store_norm(double sum, double max_norm, float* out) {
  const double norm = sqrt(sum);
  const double c = max_norm / (norm + 1e-6);
  out[0] = float(norm);
  out[1] = c >= 1.0 ? 1.0f : float(c);       // a NaN stays one
}

// Sum of squares of the elements [k0, k1) of a tensor, k0 a multiple of 8: the
// share of thread `me` of `threads`, in float64.
template <bool BF16>
__device__ __forceinline__ double square_sum(const void* g, int64_t k0, int64_t k1, int me, int threads) {
  typedef __bf16 bf16v8 __attribute__((ext_vector_type(8)));
  constexpr int E = BF16 ? 8 : 4;            // elements of a 16-byte load
  const int step = threads * E;
  double s0 = 0.0, s1 = 0.0;
  int64_t k = k0 + me * E;
  auto add = [&](const u32x4_t& raw) {
    if constexpr (BF16) {
      const bf16v8 b = __builtin_bit_cast(bf16v8, raw);
#pragma unroll
      for (int j = 0; j < 8; j += 2) {
        const double x = double(float(b[j])), y = double(float(b[j + 1]));
        s0 = __builtin_fma(x, x, s0);
        s1 = __builtin_fma(y, y, s1);
      }
    } else {
      const f32x4_t f = __builtin_bit_cast(f32x4_t, raw);
#pragma unroll
      for (int j = 0; j < 4; j += 2) {
        const double x = double(f[j]), y = double(f[j + 1]);
        s0 = __builtin_fma(x, x, s0);
        s1 = __builtin_fma(y, y, s1);
      }
    }
  };
  const u32x4_t* p = reinterpret_cast<const u32x4_t*>(g);
  // Eight loads in flight per thread. They are plain ones: with the non-temporal
  // hint this pass is faster (906 MB: 130 us against 146) but the step that
  // follows finds nothing of the gradient in the caches (norm and AdamW together
  // 1159 us against 1140).
  constexpr int U = 8;
  for (; k + (U - 1) * int64_t(step) + E <= k1; k += U * int64_t(step)) {
    u32x4_t r[U];
#pragma unroll
    for (int j = 0; j < U; ++j) r[j] = p[(k + j * int64_t(step)) / E];
#pragma unroll
    for (int j = 0; j < U; ++j) add(r[j]);
  }
  // The last vectors, four loads in flight again: those past the end repeat the
  // thread's first one and count as zeros.
  for (; k + E <= k1; k += 4 * int64_t(step)) {
    u32x4_t r[4];
    int64_t at[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      at[j] = k + j * int64_t(step);
      r[j] = p[(at[j] + E <= k1 ? at[j] : k) / E];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) add(at[j] + E <= k1 ? r[j] : u32x4_t{0u, 0u, 0u, 0u});
  }
  // The partial vector, by the thread that comes to it.
  k = k0 + (k1 - k0) / E * E;
  if ((k - k0) / E % threads != me) return s0 + s1;
  for (int64_t i = k; i < k1; ++i) {
    const double x = BF16 ? double(float(static_cast<const __bf16*>(g)[i]))
                          : double(static_cast<const float*>(g)[i]);
    s0 = __builtin_fma(x, x, s0);
  }
  return s0 + s1;
}

template <class Table>
__device__ __forceinline__ double tensor_square_sum(const Table& tab, int t, int64_t k0, int64_t k1, int me,
                                                    int threads) {
  return tab.tail[t] >> 15 ? square_sum<true>(tab.p(0, t), k0, k1, me, threads)
                           : square_sum<false>(tab.p(0, t), k0, k1, me, threads);
}

// Workgroup b sums its share of the chunks, a run of them, into part[b].
__global__ __launch_bounds__(256) void norm_partial_kernel(NormTable tab, double* part) {
  __shared__ double lds[4];
  const int per = (tab.chunks + int(gridDim.x) - 1) / int(gridDim.x);
  int c = int(blockIdx.x) * per;
  const int c1 = c + per < tab.chunks ? c + per : tab.chunks;
  double s = 0.0;
  if (c < c1) {
    for (int t = tensor_of(tab, c); c < c1; ++t) {
      const int last = (tab.first[t + 1] < c1 ? tab.first[t + 1] : c1) - 1;
      s += tensor_square_sum(tab, t, int64_t(c - tab.first[t]) * kChunk, end_of(tab, t, last),
                             int(threadIdx.x), 256);
      c = last + 1;
    }
  }
  s = block_sum(s, lds);
  if (threadIdx.x == 0) part[blockIdx.x] = s;
}

// A short list by one workgroup, a chunk to a wave at a time, and the result.
// Up to kNormAlone chunks: 4096 elements take 4.4 us, 65536 in one tensor 4.8, 60000
// in twelve 5.1-5.7, where the two launches take 5.3, 5.7 and 5.7; 131072 in one 6.9
// and 5.7.
__global__ __launch_bounds__(1024) void norm_alone_kernel(NormTable tab, double max_norm, float* out) {
  __shared__ double lds[16];
  double s = 0.0;
  for (int c = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6)); c < tab.chunks; c += 16) {
    const int t = tensor_of(tab, c);
    s += tensor_square_sum(tab, t, int64_t(c - tab.first[t]) * kChunk, end_of(tab, t, c),
                           int(threadIdx.x & 63), 64);
  }
  s = block_sum(s, lds);
  if (threadIdx.x == 0) store_norm(s, max_norm, out);
}

__global__ __launch_bounds__(1024) void norm_finish_kernel(const double* part, int64_t count,
                                                           double max_norm, float* out) {
  __shared__ double lds[16];
  double s = 0.0;
  for (int64_t k = threadIdx.x; k < count; k += 1024) s += part[k];
  s = block_sum(s, lds);
  if (threadIdx.x == 0) store_norm(s, max_norm, out);
}

enum ClipOp : int { CLIP_SCALE = 0, CLIP_ADAMW = 1, CLIP_ADAMW_EXACT = 2, CLIP_SGDM = 3 };

// One chunk of one tensor per workgroup: 4 groups of 4 elements per thread.
// Everything is read and written once, so loads and stores carry the
// non-temporal hint (AdamW on 226M elements: 5.8 TB/s against 5.4 without).
template <int OP, bool BF16, class Table>
__device__ __forceinline__ void clip_chunk(const Table& tab, int t, int c, float coef,
                                           const AdamWConsts& ac, const SgdmConsts& sc) {
  constexpr bool ADAM = OP == CLIP_ADAMW || OP == CLIP_ADAMW_EXACT;
  constexpr int G = kChunk / (256 * 4);
  const void* const g_ = tab.p(0, t);
  float* const W = static_cast<float*>(tab.p(1, t));
  float* const m = OP == CLIP_SCALE ? nullptr : static_cast<float*>(tab.p(Table::A > 2 ? 2 : 0, t));
  float* const v = ADAM ? static_cast<float*>(tab.p(Table::A > 3 ? 3 : 0, t)) : nullptr;
  const int64_t k0 = int64_t(c - tab.first[t]) * kChunk, n = end_of(tab, t, c);
  const int64_t k = k0 + int(threadIdx.x) * 4;
  auto get4 = [](const float* p) {
    return __builtin_nontemporal_load(reinterpret_cast<const f32x4_t*>(p));
  };
  auto set4 = [](float* p, const f32x4_t& x) {
    __builtin_nontemporal_store(x, reinterpret_cast<f32x4_t*>(p));
  };
  auto grad4 = [&](int64_t i) {
    if constexpr (BF16)
      return unpack_bf16x4(__builtin_nontemporal_load(
          reinterpret_cast<const u32x2_t*>(static_cast<const uint16_t*>(g_) + i)));
    else
      return get4(static_cast<const float*>(g_) + i);
  };
  if (k0 + kChunk == n) {
    f32x4_t g[G], w[G], a[G], b[G];
#pragma unroll
    for (int j = 0; j < G; ++j) {
      g[j] = grad4(k + j * 1024);
      if constexpr (OP != CLIP_SCALE) {
        w[j] = get4(W + k + j * 1024);
        a[j] = get4(m + k + j * 1024);
      }
      if constexpr (ADAM) b[j] = get4(v + k + j * 1024);
    }
#pragma unroll
    for (int j = 0; j < G; ++j) {
      g[j] = g[j] * coef;
      if constexpr (OP == CLIP_SCALE) {
        if constexpr (BF16)
          __builtin_nontemporal_store(pack_bf16x4(g[j]), reinterpret_cast<u32x2_t*>(
                                                             reinterpret_cast<uint16_t*>(W) + k + j * 1024));
        else
          set4(W + k + j * 1024, g[j]);
      } else {
        if constexpr (ADAM)
          adamw_vec4<OP == CLIP_ADAMW_EXACT>(g[j], w[j], a[j], b[j], ac);
        else
          sgdm_vec4(g[j], w[j], a[j], sc);
        set4(W + k + j * 1024, w[j]);
        set4(m + k + j * 1024, a[j]);
        if constexpr (ADAM) set4(v + k + j * 1024, b[j]);
      }
    }
    return;
  }
  // A tensor's last chunk: element by element, neighbouring lanes on
  // neighbouring elements.
  for (int64_t i = k0 + threadIdx.x; i < n; i += 256) {
    const float g = (BF16 ? float(static_cast<const __bf16*>(g_)[i]) : static_cast<const float*>(g_)[i]) * coef;
    if constexpr (OP == CLIP_SCALE) {
      if constexpr (BF16)
        reinterpret_cast<__bf16*>(W)[i] = __bf16(g);
      else
        W[i] = g;
    } else {
      float w = W[i], a = m[i];
      if constexpr (ADAM) {
        float b = v[i];
        adamw_elem<OP == CLIP_ADAMW_EXACT>(g, w, a, b, ac);
        v[i] = b;
      } else {
        sgdm_elem(g, w, a, sc);
      }
      W[i] = w;
      m[i] = a;
    }
  }
}

template <int OP, class Table>
__global__ __launch_bounds__(256) void clip_step_kernel(Table tab, const float* coef_,
                                                        AdamWConsts ac, SgdmConsts sc) {
  const float coef = *coef_;
  const int c = blockIdx.x, t = tensor_of(tab, c);
  if (tab.tail[t] >> 15)
    clip_chunk<OP, true>(tab, t, c, coef, ac, sc);
  else
    clip_chunk<OP, false>(tab, t, c, coef, ac, sc);
}

}  // namespace forge
