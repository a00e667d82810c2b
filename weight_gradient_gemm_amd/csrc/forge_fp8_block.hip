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

// Most workgroups that quantise along rows alone; what is beyond loops.
constexpr int64_t kMaxRowGroups = int64_t(1) << 20;

using Fp8128x64 = SmallTileCfg<128, 64, 2, 2, 1, 2>;
using Fp864x64 = SmallTileCfg<64, 64, 2, 2, 2, 2>;

// The library's choice of tile: the least estimated time in microseconds, from
// times measured on this kernel. A stage (64 columns) of a tile takes `alone`
// where its CU has nothing else to do, and a CU with `slots` of them finishes one
// every `full`; `ends` is what a round of tiles adds at its two ends. The
// persistent schedule runs 256x256 tiles, its rounds counted in full tiles. Of
// 35 sizes from 64 x 64 x 128 to 16384 x 6144 x 4096 one is 15% behind the fastest
// tile and the others within 10% (333 x 520 x 1024: 4.7 us at 64x64, 5.8 to 14 at the others;
// 1024 x 4096 x 4096: 17.8 at 128x128, 22 to 36; 8192 x 4096 x 14336: 312 at 256x256,
// 318 by the persistent schedule; 4096 x 6144 x 16384: 276 by that, 297 at 256x256).
//
// Up to 64 rows take the kernel that cuts the contraction where 64x64 tiles are few:
// up to so many workgroups of it (16 rows of the long operand each) to a CU as its reads of the
// short operand leave room for, three for up to 4 rows, two for up to 16, one for more. Beyond
// that tiles fill the chip as well and read the short operand less often (rows and tiles, us:
// 1 x 4096 x 14336 11.8 and 24.3; 4 x 12288 x 14336 31.4 and 35.2, x 1024 5.5 and 5.3; 4 x 14336 x 14336
// 40.2 and 36.7; 16 x 8192 x 4096 9.1 and 9.6, 16 x 9216 x 4096 10.2 and 9.7, x 14336 35.3 and 32.0; 32 x
// 4096 x 4096 6.9 and 9.8, 32 x 5120 x 4096 9.8 and 9.6; 64 x 4096 x 14336 23.2 and 24.4, x 1024 5.5 and
// 5.2, 64 x 5120 x 4096 14.4 and 9.7; 16 x 128256 x 4096 117 and 89, one row of it 92 and 92).
forge_tile choose_tile(int64_t N, int64_t M, int64_t Kp) {
  struct Kind {
    forge_tile id;
    int bm, bn, slots, ring;       // ring: stages of a round of its LDS slots
    double alone, full, ends;
  };
  static const Kind kinds[] = {{FORGE_TILE_256x256, 256, 256, 1, 4, 0.447, 0.667, 7.2},
                               {FORGE_TILE_256x128, 256, 128, 1, 4, 0.30, 0.375, 4.9},
                               {FORGE_TILE_128x128, 128, 128, 2, 4, 0.19, 0.215, 3.1},
                               {FP8_TILE_128x64, 128, 64, 1, 8, 0.136, 0.17, 3.2},
                               {FP8_TILE_64x64, 64, 64, 2, 8, 0.096, 0.10, 2.4}};
  const int64_t per_cu = M <= 4 ? 3 : M <= 16 ? 2 : M <= 64 ? 1 : 0;
  if (N <= per_cu * 256 * 16) return FP8_TILE_ROWS;
  auto stages = [&](int ring) { return double((Kp / 64 + ring - 1) / ring * ring); };
  auto round = [&](const Kind& k, int64_t tiles) {
    if (tiles == 0) return 0.0;
    const double load = double(tiles) / 256.0;
    return stages(k.ring) * std::max(k.alone, (load <= 1.0 ? load : std::ceil(load)) * k.full) + k.ends;
  };
  forge_tile best = FORGE_TILE_256x256;
  double least = 0.0;
  for (const Kind& k : kinds) {
    const int64_t tiles = count_tiles(N, M, TileShape{k.bm, k.bn}), slots = 256 * k.slots;
    const double t = double(tiles / slots) * round(k, slots) + round(k, tiles % slots);
    if (least == 0.0 || t < least) {
      least = t;
      best = k.id;
    }
  }
  const int grid = persistent_grid();
  const int64_t tiles = count_tiles(N, M, TileShape{256, 256});
  if (grid > 0 && tiles >= grid) {
    const double t = persistent_makespan(tiles, grid) * (stages(4) * 0.645 + 7.0);
    if (t < least) {
      least = t;
      best = FORGE_TILE_PERSISTENT;
    }
  }
  return best;
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
  if (a.d_out <= 16) return launch_rows_t<1, 8, 2, FI, FO>(a, x, s);
  if (a.d_out <= 32) return launch_rows_t<2, 8, 2, FI, FO>(a, x, s);
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
  if (a.col_codes) return quantize_fp8_block_kernel<BF16, E5M2, true, true>;
  return a.square ? quantize_fp8_block_kernel<BF16, E5M2, true, false> : quantize_fp8_block_rows_kernel<BF16, E5M2>;
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
  const int64_t rows = row_codes && !col_codes && !square ? kFp8RowsOf : kFp8Tile;    // of a workgroup
  const int64_t across = (C + kFp8Tile - 1) / kFp8Tile, tiles = (R + rows - 1) / rows * across;
  if (tiles >= int64_t(1) << 31) return FORGE_ERR_SHAPE;
  a.tiles = uint32_t(tiles);
  a.tiles_c = uint32_t(across);
  const bool bf16 = x_dtype == FORGE_BF16;
  const auto kernel = fmt == FORGE_FP8_E5M2 ? (bf16 ? quantize_kernel<true, true>(a) : quantize_kernel<false, true>(a))
                                            : (bf16 ? quantize_kernel<true, false>(a) : quantize_kernel<false, false>(a));
  hipLaunchKernelGGL(kernel, dim3(uint32_t(rows == kFp8Tile ? tiles : std::min(tiles, kMaxRowGroups))),
                     dim3(kFp8QuantThreads), 0,
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
  if (tile == FORGE_TILE_DEFAULT) tile = choose_tile(N, M, Kp);
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
