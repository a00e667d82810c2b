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

// The lanes at a distance: 1 and 2 within four, mirrored within 8 and within 16, and
// the value of the other row of 16, or half of the wave. Vector instructions of 4
// cycles each, where a shuffle through LDS takes some 100 (layer norm of 16384 x 4096
// bf16: 49 us, 56 by shuffles; of one row 2.3 and 2.7).
template <int CTRL>
__device__ __forceinline__ uint32_t lanes_dpp(uint32_t v) {
  return uint32_t(__builtin_amdgcn_update_dpp(0, int(v), CTRL, 0xf, 0xf, true));
}
template <int CTRL>
__device__ __forceinline__ float lanes_dpp(float v) {
  return __builtin_bit_cast(float, lanes_dpp<CTRL>(__builtin_bit_cast(uint32_t, v)));
}
template <int CTRL>
__device__ __forceinline__ double lanes_dpp(double v) {
  const u32x2_t w = __builtin_bit_cast(u32x2_t, v);
  return __builtin_bit_cast(double, u32x2_t{lanes_dpp<CTRL>(w[0]), lanes_dpp<CTRL>(w[1])});
}
// Both rows' (halves') values, the even row's (lower half's) first: a swap of a value with itself.
template <int D>
__device__ __forceinline__ void lanes_pair(uint32_t v, uint32_t& a, uint32_t& b) {
  static_assert(D == 16 || D == 32);
  if constexpr (D == 16) {
    const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
    a = r[0];
    b = r[1];
  } else {
    const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
    a = r[0];
    b = r[1];
  }
}
template <int D>
__device__ __forceinline__ void lanes_pair(float v, float& a, float& b) {
  uint32_t x, y;
  lanes_pair<D>(__builtin_bit_cast(uint32_t, v), x, y);
  a = __builtin_bit_cast(float, x);
  b = __builtin_bit_cast(float, y);
}
template <int D>
__device__ __forceinline__ void lanes_pair(double v, double& a, double& b) {
  const u32x2_t w = __builtin_bit_cast(u32x2_t, v);
  uint32_t x0, y0, x1, y1;
  lanes_pair<D>(w[0], x0, y0);
  lanes_pair<D>(w[1], x1, y1);
  a = __builtin_bit_cast(double, u32x2_t{x0, x1});
  b = __builtin_bit_cast(double, u32x2_t{y0, y1});
}

// op over the 16 lanes of a row of lanes, and over the wave, in every lane.
template <class T, class Op>
__device__ __forceinline__ T row16_all(T v, Op op) {
  v = op(v, lanes_dpp<0xB1>(v));
  v = op(v, lanes_dpp<0x4E>(v));
  v = op(v, lanes_dpp<0x141>(v));
  return op(v, lanes_dpp<0x140>(v));
}
template <class T, class Op>
__device__ __forceinline__ T rows_all(T v, Op op) {
  T a, b;
  lanes_pair<16>(v, a, b);
  v = op(a, b);
  lanes_pair<32>(v, a, b);
  return op(a, b);
}
template <class T>
__device__ __forceinline__ T wave_sum(T v) {
  const auto add = [](T x, T y) { return x + y; };
  return rows_all(row16_all(v, add), add);
}
__device__ __forceinline__ float wave_max(float v) {
  const auto larger = [](float x, float y) { return fmaxf(x, y); };
  return rows_all(row16_all(v, larger), larger);
}

}  // namespace forge
