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
constexpr int kNormTensors = 128;
constexpr int kStepTensors = 72;
constexpr int kNormChunk = 16384;    // elements of a chunk of the norm's pass
constexpr int kNormGrid = 2048;      // most workgroups (and partial sums) of a norm launch
constexpr int kStepChunk = 4096;     // elements of a chunk of the step's pass

struct NormTable {
  const void* g[kNormTensors];
  int64_t n[kNormTensors];
  int32_t first[kNormTensors];       // first chunk of tensor t; INT32_MAX past the last tensor
  uint8_t bf16[kNormTensors];
  int32_t chunks;
};

struct StepTable {
  const void* g[kStepTensors];
  void* W[kStepTensors];             // the clipped gradient's place in forge_clip_grads
  float* m[kStepTensors];
  float* v[kStepTensors];
  int64_t n[kStepTensors];
  int32_t first[kStepTensors];
  uint8_t bf16[kStepTensors];
  int32_t chunks;
};
static_assert(sizeof(NormTable) <= 4000 && sizeof(StepTable) <= 4000, "kernel argument size");

// The tensor of chunk c: the last one that starts at or before it. Every lane
// of the wave takes part.
template <int N>
__device__ __forceinline__ int tensor_of(const int32_t (&first)[N], int c) {
  const int lane = threadIdx.x & 63;
  int t = -1;
#pragma unroll
  for (int k = 0; k < N; k += 64) {
    const bool below = k + lane < N && first[k + lane < N ? k + lane : N - 1] <= c;
    t += __popcll(__ballot(below));
  }
  return __builtin_amdgcn_readfirstlane(t);
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

// Sum of squares of the elements [k0, k1) of a tensor by the workgroup, k0 a
// multiple of 8: each thread's share, in float64.
template <bool BF16>
__device__ __forceinline__ double square_sum(const void* g, int64_t k0, int64_t k1) {
  typedef __bf16 bf16v8 __attribute__((ext_vector_type(8)));
  constexpr int E = BF16 ? 8 : 4;            // elements of a 16-byte load
  const int step = int(blockDim.x) * E;
  double s0 = 0.0, s1 = 0.0;
  int64_t k = k0 + int(threadIdx.x) * E;
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
  // Four loads in flight per thread.
  for (; k + 3 * int64_t(step) + E <= k1; k += 4 * int64_t(step)) {
    u32x4_t r[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) r[j] = p[(k + j * int64_t(step)) / E];
#pragma unroll
    for (int j = 0; j < 4; ++j) add(r[j]);
  }
  for (; k + E <= k1; k += step) add(p[k / E]);
  for (int64_t i = k; i < k1; ++i) {         // the thread that owns the partial vector
    const double x = BF16 ? double(float(static_cast<const __bf16*>(g)[i]))
                          : double(static_cast<const float*>(g)[i]);
    s0 = __builtin_fma(x, x, s0);
  }
  return s0 + s1;
}

// Workgroup b sums chunks b, b + grid, ... into part[b].
__global__ __launch_bounds__(256) void norm_partial_kernel(NormTable tab, double* part) {
  __shared__ double lds[16];
  double s = 0.0;
  for (int c = blockIdx.x; c < tab.chunks; c += gridDim.x) {
    const int t = tensor_of(tab.first, c);
    const int64_t k0 = int64_t(c - tab.first[t]) * kNormChunk;
    const int64_t n = tab.n[t], k1 = k0 + kNormChunk < n ? k0 + kNormChunk : n;
    s += tab.bf16[t] ? square_sum<true>(tab.g[t], k0, k1) : square_sum<false>(tab.g[t], k0, k1);
  }
  s = block_sum(s, lds);
  if (threadIdx.x == 0) part[blockIdx.x] = s;
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
template <int OP, bool BF16>
__device__ __forceinline__ void clip_chunk(const StepTable& tab, int t, int64_t k0, float coef,
                                           const AdamWConsts& ac, const SgdmConsts& sc) {
  typedef __bf16 bf16v4 __attribute__((ext_vector_type(4)));
  constexpr bool ADAM = OP == CLIP_ADAMW || OP == CLIP_ADAMW_EXACT;
  constexpr int G = kStepChunk / (256 * 4);
  const int64_t n = tab.n[t];
  const void* const g_ = tab.g[t];
  float* const W = static_cast<float*>(tab.W[t]);
  float* const m = tab.m[t];
  float* const v = tab.v[t];
  const int64_t k = k0 + int(threadIdx.x) * 4;
  auto grad4 = [&](int64_t i) {
    if constexpr (BF16)
      return __builtin_convertvector(*reinterpret_cast<const bf16v4*>(static_cast<const __bf16*>(g_) + i),
                                     f32x4_t);
    else
      return *reinterpret_cast<const f32x4_t*>(static_cast<const float*>(g_) + i);
  };
  auto put4 = [&](int64_t i, const f32x4_t& g) {
    if constexpr (BF16)
      *reinterpret_cast<bf16v4*>(reinterpret_cast<__bf16*>(W) + i) = __builtin_convertvector(g, bf16v4);
    else
      *reinterpret_cast<f32x4_t*>(W + i) = g;
  };
  if (k0 + kStepChunk <= n) {
    f32x4_t g[G], w[G], a[G], b[G];
#pragma unroll
    for (int j = 0; j < G; ++j) {
      g[j] = grad4(k + j * 1024);
      if constexpr (OP != CLIP_SCALE) {
        w[j] = *reinterpret_cast<const f32x4_t*>(W + k + j * 1024);
        a[j] = *reinterpret_cast<const f32x4_t*>(m + k + j * 1024);
      }
      if constexpr (ADAM) b[j] = *reinterpret_cast<const f32x4_t*>(v + k + j * 1024);
    }
#pragma unroll
    for (int j = 0; j < G; ++j) {
      g[j] = g[j] * coef;
      if constexpr (OP == CLIP_SCALE) {
        put4(k + j * 1024, g[j]);
      } else {
        if constexpr (ADAM)
          adamw_vec4<OP == CLIP_ADAMW_EXACT>(g[j], w[j], a[j], b[j], ac);
        else
          sgdm_vec4(g[j], w[j], a[j], sc);
        *reinterpret_cast<f32x4_t*>(W + k + j * 1024) = w[j];
        *reinterpret_cast<f32x4_t*>(m + k + j * 1024) = a[j];
        if constexpr (ADAM) *reinterpret_cast<f32x4_t*>(v + k + j * 1024) = b[j];
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

template <int OP>
__global__ __launch_bounds__(256) void clip_step_kernel(StepTable tab, const float* coef_,
                                                        AdamWConsts ac, SgdmConsts sc) {
  const float coef = *coef_;
  const int t = tensor_of(tab.first, blockIdx.x);
  const int64_t k0 = int64_t(int(blockIdx.x) - tab.first[t]) * kStepChunk;
  if (tab.bf16[t])
    clip_chunk<OP, true>(tab, t, k0, coef, ac, sc);
  else
    clip_chunk<OP, false>(tab, t, k0, coef, ac, sc);
}

}  // namespace forge
