// Entry points of the forge C ABI for 8-bit operands with a scale for each block
// of 128.
#include <algorithm>
#include <cmath>

#include "forge_ops.h"
#include "fp8_block_kernels.hpp"
#include "host.hpp"
#include "validate_ops.hpp"

namespace forge {
namespace {

// Tiles of the library's own choice, beside the public ids.
enum : forge_tile { FP8_TILE_128x64 = FORGE_TILE_COUNT, FP8_TILE_64x64, FP8_TILE_ROWS };

using Fp8128x64 = SmallTileCfg<128, 64, 2, 2, 2, 1>;
using Fp864x64 = SmallTileCfg<64, 64, 2, 2, 4, 1>;

// The library's choice of tile: the largest that gives every compute unit some.
forge_tile choose_tile(int64_t N, int64_t M) {
  if (M <= 64 && N <= 131072) return FP8_TILE_ROWS;
  const int64_t tiles = count_tiles(N, M, TileShape{256, 256});
  if (persistent_grid() > 0 && tiles >= persistent_grid()) return FORGE_TILE_PERSISTENT;
  if (count_tiles(N, M, TileShape{256, 128}) >= 256) return FORGE_TILE_256x128;
  if (count_tiles(N, M, TileShape{128, 128}) >= 256) return FORGE_TILE_128x128;
  if (count_tiles(N, M, TileShape{128, 64}) >= 256) return FP8_TILE_128x64;
  return FP8_TILE_64x64;
}

template <class C, int FI, int FO>
forge_status launch_tile(WgradArgs a, const Fp8BlockArgs& x, hipStream_t s) {
  set_grid<C>(a, 1);
  hipLaunchKernelGGL((fp8_block_kernel<C, FI, FO>), dim3(a.num_tiles), dim3(C::THREADS), 0, s, a, x);
  return launch_status();
}

template <int MB, int W, int U, int FI, int FO>
forge_status launch_rows_t(const WgradArgs& a, const Fp8BlockArgs& x, hipStream_t s) {
  hipLaunchKernelGGL((fp8_block_rows_kernel<MB, W, U, FI, FO>), dim3((a.d_in + 15) / 16), dim3(64 * W), 0, s, a, x);
  return launch_status();
}

template <int FI, int FO>
forge_status launch_rows(const WgradArgs& a, const Fp8BlockArgs& x, hipStream_t s) {
  if (a.d_out <= 16) return launch_rows_t<1, 16, 4, FI, FO>(a, x, s);
  if (a.d_out <= 32) return launch_rows_t<2, 16, 2, FI, FO>(a, x, s);
  return launch_rows_t<4, 8, 2, FI, FO>(a, x, s);
}

template <int FI, int FO>
forge_status launch_product(WgradArgs a, const Fp8BlockArgs& x, forge_tile tile, hipStream_t s) {
  switch (tile) {
    case FP8_TILE_ROWS: return launch_rows<FI, FO>(a, x, s);
    case FP8_TILE_64x64: return launch_tile<Fp864x64, FI, FO>(a, x, s);
    case FP8_TILE_128x64: return launch_tile<Fp8128x64, FI, FO>(a, x, s);
    case FORGE_TILE_128x128: return launch_tile<Cfg128x128, FI, FO>(a, x, s);
    case FORGE_TILE_256x128: return launch_tile<Cfg256x128, FI, FO>(a, x, s);
    case FORGE_TILE_256x256: return launch_tile<Cfg256x256, FI, FO>(a, x, s);
    case FORGE_TILE_PERSISTENT: {
      const int grid = persistent_grid();
      if (grid <= 0) return launch_tile<Cfg256x256, FI, FO>(a, x, s);
      set_grid<Cfg256x256>(a, 1);
      hipLaunchKernelGGL((fp8_block_persistent_kernel<Cfg256x256, Cfg256x128, FI, FO>), dim3(grid),
                         dim3(Cfg256x256::THREADS), 0, s, a, x);
      return launch_status();
    }
    default: return FORGE_ERR_TILE;
  }
}

template <bool BF16, bool E5M2>
void (*quantize_kernel(const Fp8QuantArgs& a))(Fp8QuantArgs) {
  if (!a.row_codes) return quantize_fp8_block_kernel<BF16, E5M2, false, true>;
  return a.col_codes ? quantize_fp8_block_kernel<BF16, E5M2, true, true>
                     : quantize_fp8_block_kernel<BF16, E5M2, true, false>;
}

}  // namespace
}  // namespace forge

using namespace forge;

extern "C" {

FORGE_API forge_status forge_quantize_fp8_block(const void* x, forge_dtype x_dtype, int64_t R, int64_t C,
                                                forge_dtype fmt, int32_t square, void* row_codes,
                                                void* row_scales, void* col_codes, void* col_scales,
                                                void* stream) {
  if (forge_status s = validate_quantize_fp8_block(x, x_dtype, R, C, fmt, row_codes, row_scales,
                                                   col_codes, col_scales))
    return s;
  if (R == 0 || C == 0) return FORGE_OK;
  if (forge_status s = check_device()) return s;
  (void)hipGetLastError();
  Fp8QuantArgs a{};
  a.x = x;
  a.row_codes = static_cast<uint8_t*>(row_codes);
  a.row_scales = static_cast<uint8_t*>(row_scales);
  a.col_codes = static_cast<uint8_t*>(col_codes);
  a.col_scales = static_cast<uint8_t*>(col_scales);
  a.R = R;
  a.C = C;
  a.row_pitch = FORGE_FP8_BLOCK_ROWS(R);
  a.col_pitch = FORGE_FP8_BLOCK_ROWS(C);
  a.square = square != 0;
  const int64_t across = (C + kFp8Tile - 1) / kFp8Tile, tiles = (R + kFp8Tile - 1) / kFp8Tile * across;
  if (tiles >= int64_t(1) << 31) return FORGE_ERR_SHAPE;
  a.tiles_c = uint32_t(across);
  const bool bf16 = x_dtype == FORGE_BF16;
  const auto kernel = fmt == FORGE_FP8_E5M2 ? (bf16 ? quantize_kernel<true, true>(a) : quantize_kernel<false, true>(a))
                                            : (bf16 ? quantize_kernel<true, false>(a) : quantize_kernel<false, false>(a));
  hipLaunchKernelGGL(kernel, dim3(uint32_t(tiles)), dim3(kFp8QuantThreads), 0,
                     static_cast<hipStream_t>(stream), a);
  return launch_status();
}

FORGE_API forge_status forge_matmul_fp8_block(const void* a_codes, const void* a_scales, forge_dtype a_fmt,
                                              const void* b_codes, const void* b_scales, forge_dtype b_fmt,
                                              void* out, int64_t M, int64_t N, int64_t Kp,
                                              forge_tile tile, void* stream) {
  if (forge_status s = validate_matmul_fp8_block(a_codes, a_scales, a_fmt, b_codes, b_scales, b_fmt, out,
                                                 M, N, Kp, tile))
    return s;
  if (M == 0 || N == 0) return FORGE_OK;
  if (forge_status s = check_device()) return s;
  if (!grid_fits(N, M, FORGE_TILE_128x128, 1)) return FORGE_ERR_SHAPE;
  if (tile == FORGE_TILE_DEFAULT) tile = choose_tile(N, M);
  (void)hipGetLastError();
  const WgradArgs w = base_args(b_codes, a_codes, static_cast<float*>(out), nullptr, nullptr, Kp, N, M);
  const Fp8BlockArgs x{static_cast<const uint8_t*>(b_scales), static_cast<const uint8_t*>(a_scales), Kp};
  const hipStream_t s = static_cast<hipStream_t>(stream);
  constexpr int E4 = 0, E5 = 1;      // operand format codes of the instruction
  if (b_fmt == FORGE_FP8_E4M3)
    return a_fmt == FORGE_FP8_E4M3 ? launch_product<E4, E4>(w, x, tile, s) : launch_product<E4, E5>(w, x, tile, s);
  return a_fmt == FORGE_FP8_E4M3 ? launch_product<E5, E4>(w, x, tile, s) : launch_product<E5, E5>(w, x, tile, s);
}

}  // extern "C"
