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
// row lies in the registers of one wave (up to 1024 columns), of four or of
// sixteen, so it is read once; the variance is summed from the deviations,
// which no mean makes cancel. The backward pass's workgroups go from row to
// row with their columns' sums of dY n and dY in registers, store them at the
// end, and a second launch adds up the workgroups' sums in a fixed order.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

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

// Sum of v over the WAVES waves that share a row, in every thread. `part`: WAVES
// floats, which the next call but one may use again.
template <int WAVES>
__device__ __forceinline__ float row_sum(float v, float* part) {
  v = wave_sum(v);
  if constexpr (WAVES > 1) {
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int w = 0; w < WAVES; ++w) v += part[w];
  }
  return v;
}

// Workgroups: WAVES waves to a row, or four rows of a wave each.
template <int WAVES>
constexpr int ln_threads = WAVES == 1 ? 256 : 64 * WAVES;
template <int WAVES>
constexpr int ln_rows = WAVES == 1 ? 4 : 1;

// EL elements of the row to a thread.
template <bool XB, bool YB, int EL, int WAVES>
__global__ __launch_bounds__(ln_threads<WAVES>) void layernorm_kernel(LnArgs a) {
  constexpr int E = io_elems<XB, YB>, NV = EL / E, L = 64 * WAVES;
  __shared__ float part[2][WAVES];
  const int me = WAVES == 1 ? threadIdx.x & 63 : threadIdx.x;
  const int sub = WAVES == 1 ? threadIdx.x >> 6 : 0;
  const float d = float(a.d);
  for (int64_t row = int64_t(blockIdx.x) * ln_rows<WAVES> + sub; row < a.T;
       row += int64_t(gridDim.x) * ln_rows<WAVES>) {
    const int64_t base = row * a.d;
    float v[NV][E], s = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * L + me) * E;
      if (c < a.d) {
        load_elems<XB, E>(a.x, base + c, v[i]);
#pragma unroll
        for (int k = 0; k < E; ++k) s += v[i][k];
      }
    }
    const float mean = row_sum<WAVES>(s, part[0]) / d;
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if ((i * L + me) * E < a.d)
#pragma unroll
        for (int k = 0; k < E; ++k) {
          v[i][k] -= mean;
          s = __builtin_fmaf(v[i][k], v[i][k], s);
        }
    const float rstd = 1.0f / sqrtf(row_sum<WAVES>(s, part[1]) / d + a.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * L + me) * E;
      if (c < a.d) {
        float g[E], b[E] = {};
        load_f32<E>(a.gamma, c, g);
        if (a.beta) load_f32<E>(a.beta, c, b);
#pragma unroll
        for (int k = 0; k < E; ++k) v[i][k] = __builtin_fmaf(v[i][k] * rstd, g[k], b[k]);
        store_elems<YB, E>(a.out, base + c, v[i]);
      }
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
  __shared__ float part[2][WAVES];
  const float d = float(a.d);
  for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x) {
    const int64_t base = row * a.d;
    float v[E], s = 0.0f;
    for (int c = threadIdx.x * E; c < a.d; c += 1024 * E) {
      load_elems<XB, E>(a.x, base + c, v);
#pragma unroll
      for (int k = 0; k < E; ++k) s += v[k];
    }
    const float mean = row_sum<WAVES>(s, part[0]) / d;
    s = 0.0f;
    for (int c = threadIdx.x * E; c < a.d; c += 1024 * E) {
      load_elems<XB, E>(a.x, base + c, v);
#pragma unroll
      for (int k = 0; k < E; ++k) {
        const float e = v[k] - mean;
        s = __builtin_fmaf(e, e, s);
      }
    }
    const float rstd = 1.0f / sqrtf(row_sum<WAVES>(s, part[1]) / d + a.eps);
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

// dX of the workgroup's rows, and its sums of dY n and dY.
template <bool XB, bool YB, int EL, int WAVES>
__global__ __launch_bounds__(ln_threads<WAVES>) void layernorm_backward_kernel(LnArgs a) {
  constexpr int E = io_elems<XB, YB>, NV = EL / E, L = 64 * WAVES;
  __shared__ float part[2][2][WAVES];
  __shared__ __attribute__((aligned(16))) float join[WAVES == 1 ? 3 * 2 * 64 * EL : 4];
  const int me = WAVES == 1 ? threadIdx.x & 63 : threadIdx.x;
  const int sub = WAVES == 1 ? threadIdx.x >> 6 : 0;
  const float d = float(a.d);
  float dg[NV][E], db[NV][E], g[NV][E];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (i * L + me) * E;
#pragma unroll
    for (int k = 0; k < E; ++k) dg[i][k] = db[i][k] = g[i][k] = 0.0f;
    if (c < a.d) load_f32<E>(a.gamma, c, g[i]);
  }
  int turn = 0;
  for (int64_t row = int64_t(blockIdx.x) * ln_rows<WAVES> + sub; row < a.T;
       row += int64_t(gridDim.x) * ln_rows<WAVES>, turn ^= 1) {
    const int64_t base = row * a.d;
    const float mean = a.mean[row], rstd = a.rstd[row];
    float n[NV][E], y[NV][E], s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * L + me) * E;
      if (c < a.d) {
        load_elems<XB, E>(a.x, base + c, n[i]);
        load_elems<YB, E>(a.dy, base + c, y[i]);
#pragma unroll
        for (int k = 0; k < E; ++k) {
          n[i][k] = (n[i][k] - mean) * rstd;
          dg[i][k] = __builtin_fmaf(y[i][k], n[i][k], dg[i][k]);
          db[i][k] += y[i][k];
          y[i][k] *= g[i][k];
          s1 += y[i][k];
          s2 = __builtin_fmaf(y[i][k], n[i][k], s2);
        }
      }
    }
    s1 = wave_sum(s1);
    s2 = wave_sum(s2);
    if constexpr (WAVES > 1) {
      if ((threadIdx.x & 63) == 0) {
        part[turn][0][threadIdx.x >> 6] = s1;
        part[turn][1][threadIdx.x >> 6] = s2;
      }
      __syncthreads();
      s1 = s2 = 0.0f;
#pragma unroll
      for (int w = 0; w < WAVES; ++w) {
        s1 += part[turn][0][w];
        s2 += part[turn][1][w];
      }
    }
    s1 /= d;
    s2 /= d;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * L + me) * E;
      if (c < a.d) {
#pragma unroll
        for (int k = 0; k < E; ++k) y[i][k] = rstd * (y[i][k] - s1 - n[i][k] * s2);
        store_elems<XB, E>(a.out, base + c, y[i]);
      }
    }
  }
  if constexpr (WAVES == 1) {                // four waves' sums to one
    if (sub > 0) {
      float* const at = join + (sub - 1) * 2 * 64 * EL;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < E; ++k) {
          at[(i * E + k) * 64 + me] = dg[i][k];
          at[(EL + i * E + k) * 64 + me] = db[i][k];
        }
    }
    __syncthreads();
    if (sub > 0) return;
#pragma unroll
    for (int w = 0; w < 3; ++w)
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < E; ++k) {
          dg[i][k] += join[w * 2 * 64 * EL + (i * E + k) * 64 + me];
          db[i][k] += join[w * 2 * 64 * EL + (EL + i * E + k) * 64 + me];
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

// dgamma and dbeta: column c of `columns` summed over the parts, 16 lanes of 4
// columns by 16 groups that take every 16th part.
struct LnReduce {
  const float* part;
  float *dgamma, *dbeta;
  int32_t d, parts, columns;         // columns: 2 d, or d without dbeta
};
__global__ __launch_bounds__(256) void layernorm_reduce_kernel(LnReduce a) {
  __shared__ f32x4_t join[16][16];
  const int me = threadIdx.x & 15, grp = threadIdx.x >> 4;
  const int c = (blockIdx.x * 16 + me) * 4;
  f32x4_t s = {0.0f, 0.0f, 0.0f, 0.0f};
  if (c < a.columns)
    for (int p = grp; p < a.parts; p += 16)
      s = s + *reinterpret_cast<const f32x4_t*>(a.part + int64_t(p) * 2 * a.d + c);
  join[grp][me] = s;
  __syncthreads();
  if (grp > 0 || c >= a.columns) return;
  for (int k = 1; k < 16; ++k) s = s + join[k][me];
  *reinterpret_cast<f32x4_t*>(c < a.d ? a.dgamma + c : a.dbeta + (c - a.d)) = s;
}

}  // namespace forge
