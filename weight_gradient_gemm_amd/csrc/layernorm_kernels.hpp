// Layer norm over the rows of x [T, d] for gfx950, and its backward pass with
// the reduction of the weight's and the bias's gradients over the rows.
//
//   mean = sum x / d,  rstd = 1 / sqrt(sum (x - mean)^2 / d + eps)
//   y = (x - mean) rstd gamma + beta
//   n = (x - mean) rstd,  a = dY gamma
//   dX = rstd (a - sum a / d - n sum (a n) / d)
//   dgamma = sum_t dY n,  dbeta = sum_t dY
//
// About ten operations an element: bound by HBM, and by latency for few rows. A
// row lies in the registers of one wave (up to 1024 columns), of four (up to 8192) or
// of eight (up to 16384), so it is read once; longer ones are read again from the
// caches. The mean is summed in 64 bits, the variance from the deviations, which no mean
// makes cancel, in float32, and in 64 bits where their squares leave its range. The backward pass's workgroups go from row to row with their columns'
// sums of dY n and dY in registers, store them at the end, and a second launch
// adds up the workgroups' sums in a fixed order.
//
// Measured, 16384 x 4096 bf16: forward 49 us, 5.5 TB/s (a copy of 4 GiB reaches 4.8, an
// addition in place 5.9); backward 75 us, 5.4 TB/s, of which the second launch (16
// MB) 5. A row after the other with the next one's loads in flight and gamma in
// registers, against a workgroup to a row: backward 77 and 103 us (with 8 instead of 64
// groups in the second launch). Accesses past the caches (kStatePolicy): loads and
// stores 56.4 us, one of the two 57.5 and 57.8, none 59.0, when the sums over a wave
// still took 7 of them. One row of 4096 takes 2.3 us, 333 x 1000 float32 backward 4.2 + 2.7.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "row_io.hpp"

namespace forge {

struct LnArgs {
  const void *x, *dy;
  const float *gamma, *beta;
  void* out;                         // y, or dX (which may be dy)
  float *mean, *rstd;                // written by the forward pass, read by the backward pass
  float* part;                       // [parts][2][d]
  int64_t T;
  int32_t d;
  float eps;
};

// Sum of v over the WAVES waves that share a row, in every thread. `part`: a
// number for each wave, which the next call but one may use again.
template <int WAVES, class F>
__device__ __forceinline__ F row_sum(F v, F* part) {
  v = wave_sum(v);
  if constexpr (WAVES > 1) {
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = part[0];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) v += part[w];
  }
  return v;
}

// Whether a variance (with eps) was summed in float32 as it should be. Below 2^-100 squares
// count that float32 holds as denormals or not at all (each of them is off by at most 2^-150),
// and one that is no number or infinite may be a sum that passed the range. The value is
// the same in all waves of the row.
__device__ __forceinline__ bool ln_in_range(float var) {
  return __builtin_amdgcn_readfirstlane(int(var >= 0x1p-100f && var <= 0x1.fffffep127f)) != 0;
}

// 1 / sqrt(sum of squares / d + eps) in 64 bits.
__device__ __forceinline__ float ln_rstd(double squares, int d, float eps) {
  return float(1.0 / sqrt(squares / double(d) + double(eps)));
}

// Workgroups: WAVES waves to a row, or four rows of a wave each.
template <int WAVES>
constexpr int ln_threads = WAVES == 1 ? 256 : 64 * WAVES;
template <int WAVES>
constexpr int ln_rows = WAVES == 1 ? 4 : 1;

// A row's vectors as they lie in memory: thread `me` of the row's L has the
// elements (i L + me) E .. + E - 1 for each i. Those past the row's end, and all of a
// row that is not wanted, read as zeros without a memory access.
template <bool BF16, int E>
using LnRaw = typename std::conditional<BF16 && E == 4, u32x2_t, u32x4_t>::type;

template <bool BF16, int E, int NV, int L>
__device__ __forceinline__ void ln_fetch(const void* p, int64_t row, int d, bool wanted, int me,
                                         LnRaw<BF16, E> (&raw)[NV]) {
  constexpr int S = BF16 ? 2 : 4;
  const __amdgpu_buffer_rsrc_t r =
      window(static_cast<const char*>(p) + (wanted ? row * d * S : 0), wanted ? int64_t(d) * S : 0);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if constexpr (E * S == 8)
      raw[i] = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_raw_buffer_load_b64(r, me * 8, i * L * 8, kStatePolicy));
    else
      raw[i] = __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, me * 16, i * L * 16, kStatePolicy));
  }
}

template <bool BF16, int E>
__device__ __forceinline__ void ln_values(const LnRaw<BF16, E>& r, float (&v)[E]) {
#pragma unroll
  for (int k = 0; k < E; ++k)
    v[k] = __builtin_bit_cast(float, BF16 ? (k & 1 ? r[k / 2] & 0xffff0000u : r[k / 2] << 16) : r[k]);
}

// Vector i of row `row`; past the row's end nothing is written.
template <bool BF16, int E, int L>
__device__ __forceinline__ void ln_put(void* p, int64_t row, int d, int me, int i, const float (&v)[E]) {
  constexpr int S = BF16 ? 2 : 4;
  const __amdgpu_buffer_rsrc_t r = window(static_cast<char*>(p) + row * d * S, int64_t(d) * S);
  const f32x4_t lo = {v[0], v[1], v[2], v[3]};
  if constexpr (E == 8) {
    const u32x2_t a = pack_bf16x4(lo), b = pack_bf16x4(f32x4_t{v[4], v[5], v[6], v[7]});
    store16(r, uint32_t(me * 16), uint32_t(i * L * 16), u32x4_t{a[0], a[1], b[0], b[1]});
  } else {
    store4<S>(r, uint32_t(me * 4 * S), uint32_t(i * L * 4 * S), lo);
  }
}

// EL elements of the row to a thread. A workgroup goes from row to row with gamma
// and beta in registers, the next row's loads in flight.
template <bool XB, bool YB, int EL, int WAVES>
__global__ __launch_bounds__(ln_threads<WAVES>) void layernorm_kernel(LnArgs a) {
  constexpr int E = io_elems<XB, YB>, NV = EL / E, L = 64 * WAVES;
  __shared__ double part_s[WAVES], part_w[WAVES];
  __shared__ float part_v[WAVES];
  const int me = WAVES == 1 ? threadIdx.x & 63 : threadIdx.x;
  const int sub = WAVES == 1 ? __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) : 0;
  const int64_t step = int64_t(gridDim.x) * ln_rows<WAVES>;
  int64_t row = int64_t(blockIdx.x) * ln_rows<WAVES> + sub;
  LnRaw<XB, E> raw[NV];
  ln_fetch<XB, E, NV, L>(a.x, row, a.d, row < a.T, me, raw);
  float g[NV][E] = {}, b[NV][E] = {};
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * L + me) * E;
    if (c < a.d) {
      load_f32<E>(a.gamma, c, g[i]);
      if (a.beta) load_f32<E>(a.beta, c, b[i]);
    }
  }
  for (; row < a.T; row += step) {
    float v[NV][E];
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      ln_values<XB, E>(raw[i], v[i]);
#pragma unroll
      for (int k = 0; k < E; ++k) s += double(v[i][k]);
    }
    ln_fetch<XB, E, NV, L>(a.x, row + step, a.d, row + step < a.T, me, raw);
    const float mean = float(row_sum<WAVES>(s, part_s) / double(a.d));
    float q = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const bool in = (i * L + me) * E < a.d;
#pragma unroll
      for (int k = 0; k < E; ++k) {
        v[i][k] = in ? v[i][k] - mean : 0.0f;
        q = __builtin_fmaf(v[i][k], v[i][k], q);
      }
    }
    const float var = row_sum<WAVES>(q, part_v) / float(a.d) + a.eps;
    float rstd = 1.0f / sqrtf(var);
    if (!ln_in_range(var)) {
      double w = 0.0;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < E; ++k) w += double(v[i][k]) * double(v[i][k]);
      rstd = ln_rstd(row_sum<WAVES>(w, part_w), a.d, a.eps);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int k = 0; k < E; ++k) v[i][k] = __builtin_fmaf(v[i][k] * rstd, g[i][k], b[i][k]);
      ln_put<YB, E, L>(a.out, row, a.d, me, i, v[i]);
    }
    if (me == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
  }
}

// Rows of any length: read three times, the second and third time from the caches.
template <bool XB, bool YB>
__global__ __launch_bounds__(1024) void layernorm_wide_kernel(LnArgs a) {
  constexpr int E = io_elems<XB, YB>, WAVES = 16;
  __shared__ double part_s[WAVES], part_w[WAVES];
  __shared__ float part_v[WAVES];
  const float d = float(a.d);
  for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x) {
    const int64_t base = row * a.d;
    float v[E], s = 0.0f;
    double sum = 0.0;
    for (int c = threadIdx.x * E; c < a.d; c += 1024 * E) {
      load_elems<XB, E>(a.x, base + c, v);
#pragma unroll
      for (int k = 0; k < E; ++k) sum += double(v[k]);
    }
    const float mean = float(row_sum<WAVES>(sum, part_s) / double(a.d));
    for (int c = threadIdx.x * E; c < a.d; c += 1024 * E) {
      load_elems<XB, E>(a.x, base + c, v);
#pragma unroll
      for (int k = 0; k < E; ++k) {
        const float e = v[k] - mean;
        s = __builtin_fmaf(e, e, s);
      }
    }
    const float var = row_sum<WAVES>(s, part_v) / d + a.eps;
    float rstd = 1.0f / sqrtf(var);
    if (!ln_in_range(var)) {
      sum = 0.0;
      for (int c = threadIdx.x * E; c < a.d; c += 1024 * E) {
        load_elems<XB, E>(a.x, base + c, v);
#pragma unroll
        for (int k = 0; k < E; ++k) {
          const double e = double(v[k] - mean);
          sum += e * e;
        }
      }
      rstd = ln_rstd(row_sum<WAVES>(sum, part_w), a.d, a.eps);
    }
    for (int c = threadIdx.x * E; c < a.d; c += 1024 * E) {
      float g[E], b[E] = {};
      load_elems<XB, E>(a.x, base + c, v);
      load_f32<E>(a.gamma, c, g);
      if (a.beta) load_f32<E>(a.beta, c, b);
#pragma unroll
      for (int k = 0; k < E; ++k) v[k] = __builtin_fmaf((v[k] - mean) * rstd, g[k], b[k]);
      store_elems<YB, E>(a.out, base + c, v);
    }
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
  }
}

// dX of the workgroup's rows, and its sums of dY n and dY. ROWS rows at a time, WAVES
// waves to each, whose sums are joined at the end: rows of up to 1024 columns, and those of up to
// 2048, of which a CU takes more waves than the others' registers leave room for
// (32768 x 2048 bf16 82 us, 102 with a row and 512 workgroups; 16384 x 4096 with two
// rows 87, with one 79). The next rows' loads are in flight; dX may be dY, whose rows no
// other workgroup reads.
template <bool XB, bool YB, int EL, int WAVES, int ROWS>
__global__ __launch_bounds__(64 * WAVES * ROWS) void layernorm_backward_kernel(LnArgs a) {
  constexpr int E = io_elems<XB, YB>, NV = EL / E, L = 64 * WAVES;
  __shared__ float part[2][2][WAVES * ROWS];
  __shared__ float join[ROWS > 1 ? (ROWS - 1) * 2 * L * EL : 1];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int sub = wave / WAVES, me = int(threadIdx.x) - sub * L;
  const float d = float(a.d);
  const int64_t step = int64_t(gridDim.x) * ROWS;
  int64_t first = int64_t(blockIdx.x) * ROWS;
  LnRaw<XB, E> rx[NV];
  LnRaw<YB, E> ry[NV];
  float mean = 0.0f, rstd = 0.0f;
  auto fetch = [&](int64_t r) {
    const bool wanted = r < a.T;
    ln_fetch<XB, E, NV, L>(a.x, r, a.d, wanted, me, rx);
    ln_fetch<YB, E, NV, L>(a.dy, r, a.d, wanted, me, ry);
    mean = wanted ? a.mean[r] : 0.0f;
    rstd = wanted ? a.rstd[r] : 0.0f;
  };
  fetch(first + sub);
  // gamma stays in registers where there is room; else it comes from the caches.
  constexpr bool HELD = EL <= 16;
  float dg[NV][E] = {}, db[NV][E] = {}, held[HELD ? NV : 1][E] = {};
  if constexpr (HELD)
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * L + me) * E;
      if (c < a.d) load_f32<E>(a.gamma, c, held[i]);
    }
  const __amdgpu_buffer_rsrc_t gammas = window(a.gamma, int64_t(a.d) * 4);
  int turn = 0;
  // Waves that wait for each other have the same number of rounds.
  for (; WAVES == 1 ? first + sub < a.T : first < a.T; first += step, turn ^= 1) {
    const int64_t row = first + sub;
    // Past the row's end, and in a row past the last, dY is 0, and so is all that it is
    // multiplied with.
    float n[NV][E], y[NV][E], s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      ln_values<XB, E>(rx[i], n[i]);
      ln_values<YB, E>(ry[i], y[i]);
      const bool in = (i * L + me) * E < a.d;
      float g[E];
      if constexpr (HELD) {
#pragma unroll
        for (int k = 0; k < E; ++k) g[k] = held[i][k];
      } else {
#pragma unroll
        for (int j = 0; j < E; j += 4) {
          const f32x4_t r = __builtin_bit_cast(f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(
              gammas, me * E * 4 + j * 4, i * L * E * 4, 0));
#pragma unroll
          for (int k = 0; k < 4; ++k) g[j + k] = r[k];
        }
      }
#pragma unroll
      for (int k = 0; k < E; ++k) {
        n[i][k] = in ? (n[i][k] - mean) * rstd : 0.0f;
        dg[i][k] = __builtin_fmaf(y[i][k], n[i][k], dg[i][k]);
        db[i][k] += y[i][k];
        y[i][k] *= g[k];
        s1 += y[i][k];
        s2 = __builtin_fmaf(y[i][k], n[i][k], s2);
      }
    }
    const float r = rstd;
    fetch(row + step);
    s1 = wave_sum(s1);
    s2 = wave_sum(s2);
    if constexpr (WAVES > 1) {
      if ((threadIdx.x & 63) == 0) {
        part[turn][0][wave] = s1;
        part[turn][1][wave] = s2;
      }
      __syncthreads();
      s1 = s2 = 0.0f;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) {
        s1 += part[turn][0][sub * WAVES + w];
        s2 += part[turn][1][sub * WAVES + w];
      }
    }
    s1 /= d;
    s2 /= d;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int k = 0; k < E; ++k) y[i][k] = r * (y[i][k] - s1 - n[i][k] * s2);
      if (WAVES == 1 || ROWS == 1 || row < a.T) ln_put<XB, E, L>(a.out, row, a.d, me, i, y[i]);
    }
  }
  if constexpr (ROWS > 1) {                  // the rows' sums to one
    if (sub > 0) {
      float* const at = join + (sub - 1) * 2 * L * EL;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < E; ++k) {
          at[(i * E + k) * L + me] = dg[i][k];
          at[(EL + i * E + k) * L + me] = db[i][k];
        }
    }
    __syncthreads();
    if (sub > 0) return;
#pragma unroll
    for (int w = 0; w < ROWS - 1; ++w)
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < E; ++k) {
          dg[i][k] += join[w * 2 * L * EL + (i * E + k) * L + me];
          db[i][k] += join[w * 2 * L * EL + (EL + i * E + k) * L + me];
        }
  }
  float* const out = a.part + int64_t(blockIdx.x) * 2 * a.d;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * L + me) * E;
    if (c < a.d)
#pragma unroll
      for (int j = 0; j < E; j += 4) {
        *reinterpret_cast<f32x4_t*>(out + c + j) = f32x4_t{dg[i][j], dg[i][j + 1], dg[i][j + 2], dg[i][j + 3]};
        *reinterpret_cast<f32x4_t*>(out + a.d + c + j) =
            f32x4_t{db[i][j], db[i][j + 1], db[i][j + 2], db[i][j + 3]};
      }
  }
}

// dX alone, of rows of any length: read twice, the second time from the caches.
template <bool XB, bool YB>
__global__ __launch_bounds__(1024) void layernorm_dx_wide_kernel(LnArgs a) {
  constexpr int E = io_elems<XB, YB>, WAVES = 16;
  __shared__ float part[2][WAVES];
  const float d = float(a.d);
  for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x) {
    const int64_t base = row * a.d;
    const float mean = a.mean[row], rstd = a.rstd[row];
    float n[E], y[E], g[E], s1 = 0.0f, s2 = 0.0f;
    for (int c = threadIdx.x * E; c < a.d; c += 1024 * E) {
      load_elems<XB, E>(a.x, base + c, n);
      load_elems<YB, E>(a.dy, base + c, y);
      load_f32<E>(a.gamma, c, g);
#pragma unroll
      for (int k = 0; k < E; ++k) {
        const float v = y[k] * g[k];
        s1 += v;
        s2 = __builtin_fmaf(v, (n[k] - mean) * rstd, s2);
      }
    }
    s1 = row_sum<WAVES>(s1, part[0]) / d;
    s2 = row_sum<WAVES>(s2, part[1]) / d;
    for (int c = threadIdx.x * E; c < a.d; c += 1024 * E) {
      load_elems<XB, E>(a.x, base + c, n);
      load_elems<YB, E>(a.dy, base + c, y);
      load_f32<E>(a.gamma, c, g);
#pragma unroll
      for (int k = 0; k < E; ++k) y[k] = rstd * (y[k] * g[k] - s1 - (n[k] - mean) * rstd * s2);
      store_elems<XB, E>(a.out, base + c, y);
    }
  }
}

// The sums of dY n and dY over the rows of a part (blockIdx.y): 32 vectors of
// columns by 8 rows at a time.
constexpr int kLnColumnRows = 8;
template <bool XB, bool YB>
__global__ __launch_bounds__(256) void layernorm_columns_kernel(LnArgs a) {
  constexpr int E = io_elems<XB, YB>;
  __shared__ float join[2][E][256];
  const int me = threadIdx.x & 31, sub = threadIdx.x >> 5;
  const int c = (blockIdx.x * 32 + me) * E;
  float dg[E] = {}, db[E] = {};
  if (c < a.d)
    for (int64_t row = int64_t(blockIdx.y) * kLnColumnRows + sub; row < a.T;
         row += int64_t(gridDim.y) * kLnColumnRows) {
      const float mean = a.mean[row], rstd = a.rstd[row];
      float n[E], y[E];
      load_elems<XB, E>(a.x, row * a.d + c, n);
      load_elems<YB, E>(a.dy, row * a.d + c, y);
#pragma unroll
      for (int k = 0; k < E; ++k) {
        dg[k] = __builtin_fmaf(y[k], (n[k] - mean) * rstd, dg[k]);
        db[k] += y[k];
      }
    }
#pragma unroll
  for (int k = 0; k < E; ++k) {
    join[0][k][threadIdx.x] = dg[k];
    join[1][k][threadIdx.x] = db[k];
  }
  __syncthreads();
  if (sub > 0 || c >= a.d) return;
  float* const out = a.part + int64_t(blockIdx.y) * 2 * a.d + c;
#pragma unroll
  for (int k = 0; k < E; ++k) {
    for (int w = 1; w < kLnColumnRows; ++w) {
      dg[k] += join[0][k][w * 32 + me];
      db[k] += join[1][k][w * 32 + me];
    }
    out[k] = dg[k];
    out[a.d + k] = db[k];
  }
}

// dgamma and dbeta: column c of `columns` summed over the parts, 8 lanes of 4
// columns (a line) by 64 groups that take every 64th part. In 64 bits, so that up to 512
// sums are joined with one rounding.
struct LnReduce {
  const float* part;
  float *dgamma, *dbeta;
  int32_t d, parts, columns;         // columns: 2 d, or d without dbeta
};
constexpr int kLnReduceColumns = 32, kLnReduceGroups = 64;
__global__ __launch_bounds__(512) void layernorm_reduce_kernel(LnReduce a) {
  __shared__ double join[kLnReduceGroups][kLnReduceColumns + 1];
  const int me = threadIdx.x & 7, grp = threadIdx.x >> 3;
  const int c = blockIdx.x * kLnReduceColumns + me * 4;
  double s[4] = {0.0, 0.0, 0.0, 0.0};
  if (c < a.columns) {
    const float* p = a.part + c;
    const int64_t step = int64_t(kLnReduceGroups) * 2 * a.d;
    f32x4_t v[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {              // at most kLayernormParts = 512 parts
      const bool in = grp + k * kLnReduceGroups < a.parts;
      v[k] = in ? *reinterpret_cast<const f32x4_t*>(p + int64_t(grp) * 2 * a.d + k * step)
                : f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    }
#pragma unroll
    for (int k = 0; k < 8; ++k)
#pragma unroll
      for (int j = 0; j < 4; ++j) s[j] += double(v[k][j]);
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) join[grp][me * 4 + j] = s[j];
  __syncthreads();
  // Eight lanes to a column, each with eight groups.
  if (threadIdx.x >= 8 * kLnReduceColumns) return;
  const int at = threadIdx.x >> 3, col = blockIdx.x * kLnReduceColumns + at;
  double r = 0.0;
#pragma unroll
  for (int k = 0; k < kLnReduceGroups / 8; ++k) r += join[me * (kLnReduceGroups / 8) + k][at];
  r += lanes_dpp<0xB1>(r);
  r += lanes_dpp<0x4E>(r);
  r += lanes_dpp<0x141>(r);
  if (me == 0 && col < a.columns) (col < a.d ? a.dgamma + col : a.dbeta + (col - a.d))[0] = float(r);
}

}  // namespace forge
