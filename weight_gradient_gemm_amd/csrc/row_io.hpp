// Vector accesses to float32 and bf16 rows, and sums over a wave, of the kernels
// that go through rows.
#pragma once

#include "wgrad_kernels.hpp"

namespace forge {

// Elements of a vector access: 16 bytes of the wider type.
template <bool XB, bool YB>
constexpr int io_elems = XB && YB ? 8 : 4;

// E consecutive elements of a float32 or bf16 array.
template <bool BF16, int E>
__device__ __forceinline__ void load_elems(const void* p, int64_t at, float (&v)[E]) {
  if constexpr (BF16 && E == 8) {
    const u32x4_t r = *reinterpret_cast<const u32x4_t*>(static_cast<const uint16_t*>(p) + at);
    const f32x4_t lo = unpack_bf16x4(u32x2_t{r[0], r[1]}), hi = unpack_bf16x4(u32x2_t{r[2], r[3]});
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      v[k] = lo[k];
      v[4 + k] = hi[k];
    }
  } else {
    const f32x4_t r = BF16 ? unpack_bf16x4(*reinterpret_cast<const u32x2_t*>(static_cast<const uint16_t*>(p) + at))
                           : *reinterpret_cast<const f32x4_t*>(static_cast<const float*>(p) + at);
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = r[k];
  }
}

template <bool BF16, int E>
__device__ __forceinline__ void store_elems(void* p, int64_t at, const float (&v)[E]) {
  if constexpr (BF16 && E == 8) {
    const u32x2_t lo = pack_bf16x4(f32x4_t{v[0], v[1], v[2], v[3]});
    const u32x2_t hi = pack_bf16x4(f32x4_t{v[4], v[5], v[6], v[7]});
    *reinterpret_cast<u32x4_t*>(static_cast<uint16_t*>(p) + at) = u32x4_t{lo[0], lo[1], hi[0], hi[1]};
  } else {
    const f32x4_t r = {v[0], v[1], v[2], v[3]};
    if constexpr (BF16)
      *reinterpret_cast<u32x2_t*>(static_cast<uint16_t*>(p) + at) = pack_bf16x4(r);
    else
      *reinterpret_cast<f32x4_t*>(static_cast<float*>(p) + at) = r;
  }
}

// E consecutive elements of a float32 array.
template <int E>
__device__ __forceinline__ void load_f32(const float* p, int64_t at, float (&v)[E]) {
#pragma unroll
  for (int j = 0; j < E; j += 4) {
    const f32x4_t r = *reinterpret_cast<const f32x4_t*>(p + at + j);
#pragma unroll
    for (int k = 0; k < 4; ++k) v[j + k] = r[k];
  }
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor(v, d));
  return v;
}

}  // namespace forge
