// Rows and units of the embedding kernels: index arithmetic with a 32-bit division
// for all but the largest arrays, for the device and for the host, where the
// tests compare it with the plain division.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace forge {

// Work in units of a few columns, counted through all rows on end: workgroups
// of 256 units then write whole lines and have no idle threads, whatever d is.
// (With a workgroup to a row, or a slice of one, 112822 rows of 1384 float32
// were written at 4.5 TB/s, rows of 1024 at 7.2.)
struct Rows {
  uint32_t units;      // of a row
  uint32_t magic;      // ceil(2^20 / units), for units < 256
};

// Row and unit of place q < units + 256 of row `row`. Fewer than 512 units are
// divided by multiplying: units * 512 < 2^20 makes it exact.
__host__ __device__ __forceinline__ void carry(const Rows& r, uint32_t q, uint32_t& row, uint32_t& unit) {
  const uint32_t over = r.units >= 256 ? uint32_t(q >= r.units) : (q * r.magic) >> 20;
  row += over;
  unit = q - over * r.units;
}

// Row and unit of the thread `tid` < 256 behind `first` units.
__host__ __device__ __forceinline__ void locate(const Rows& r, uint64_t first, uint32_t tid,
                                                uint32_t& row, uint32_t& unit) {
  row = first >> 32 ? uint32_t(first / r.units) : uint32_t(first) / r.units;
  carry(r, uint32_t(first - uint64_t(row) * r.units) + tid, row, unit);
}

}  // namespace forge
