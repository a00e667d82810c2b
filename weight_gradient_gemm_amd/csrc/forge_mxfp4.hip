// Microscaled 4-bit entry points of the forge C ABI.
#include <algorithm>
#include <cmath>

#include "forge_ops.h"
#include "host.hpp"
#include "mxfp4_kernels.hpp"
#include "validate_ops.hpp"

namespace forge {
namespace {

// Tiles of the library's own choice, beside the public ids. 64x64x2: slots of
// two stages, more in flight for long contractions of few tiles.
enum : forge_tile { MX_TILE_128x64 = FORGE_TILE_COUNT, MX_TILE_64x64, MX_TILE_64x64x2 };

// The library's choice of tile: the least estimated time in microseconds, from
// times measured on this kernel. A stage (128 columns) of a tile takes `alone`
// where a CU has nothing else to do, and a CU with `slots` of them finishes one
// every `full`; `ends` is what a round of tiles adds at its two ends. The
// persistent schedule runs 256x256 tiles, its rounds counted in full tiles.
// Of 23 sizes from 64 x 1024 x 128 to 4096 x 8192 x 8192 and 1 x 4096 x 14336 one is
// 11% behind the fastest tile and the others within 6% (1024 x 4096 x 8192: 21 us at
// 128x128, 26 to 40 at the others; 1 x 4096 x 14336: 15 at 64x64 with slots of two
// stages, 16 to 61). All with a float32 store: which epilogue follows does not enter.
forge_tile choose_tile(int64_t N, int64_t M, int64_t Kp) {
  struct Kind {
    forge_tile id;
    int bm, bn, slots, ring;       // ring: stages of a round of its LDS slots
    double alone, full, ends;
  };
  static const Kind kinds[] = {{FORGE_TILE_256x256, 256, 256, 1, 4, 0.47, 0.92, 8.5},
                               {FORGE_TILE_256x128, 256, 128, 1, 4, 0.267, 0.48, 5.2},
                               {FORGE_TILE_128x128, 128, 128, 2, 4, 0.175, 0.28, 3.8},
                               {MX_TILE_128x64, 128, 64, 3, 4, 0.152, 0.17, 3.2},
                               {MX_TILE_64x64, 64, 64, 4, 4, 0.115, 0.118, 2.8},
                               {MX_TILE_64x64x2, 64, 64, 2, 8, 0.098, 0.108, 3.1}};
  auto stages = [&](int ring) { return double((Kp / 128 + ring - 1) / ring * ring); };
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
  if (grid > 0 && tiles >= grid && persistent_makespan(tiles, grid) * (stages(4) * 0.84 + 7.1) < least)
    best = FORGE_TILE_PERSISTENT;
  return best;
}

template <class C, int EPI>
forge_status launch_mx_t(WgradArgs a, const MxArgs& x, hipStream_t s) {
  set_grid<C>(a, 1);
  hipLaunchKernelGGL((mxfp4_kernel<C, EPI>), dim3(a.num_tiles), dim3(C::THREADS), 0, s, a, x);
  return launch_status();
}

template <int EPI>
struct MxLaunch {
  static forge_status run(WgradArgs a, const MxArgs& x, forge_tile tile, hipStream_t s) {
    switch (tile) {
      case MX_TILE_64x64: return launch_mx_t<Mx64x64, EPI>(a, x, s);
      case MX_TILE_64x64x2: return launch_mx_t<Mx64x64x2, EPI>(a, x, s);
      case MX_TILE_128x64: return launch_mx_t<Mx128x64, EPI>(a, x, s);
      case FORGE_TILE_128x128: return launch_mx_t<Cfg128x128, EPI>(a, x, s);
      case FORGE_TILE_256x128: return launch_mx_t<Cfg256x128, EPI>(a, x, s);
      case FORGE_TILE_256x256: return launch_mx_t<Cfg256x256, EPI>(a, x, s);
      case FORGE_TILE_PERSISTENT: {
        const int grid = persistent_grid();
        if (grid <= 0) return launch_mx_t<Cfg256x256, EPI>(a, x, s);
        set_grid<Cfg256x256>(a, 1);
        hipLaunchKernelGGL((mxfp4_persistent_kernel<Cfg256x256, Cfg256x128, EPI>), dim3(grid),
                           dim3(Cfg256x256::THREADS), 0, s, a, x);
        return launch_status();
      }
      default: return FORGE_ERR_TILE;
    }
  }
};

template <bool BF16>
void (*quantize_kernel(const QuantArgs& a))(QuantArgs) {
  if (!a.row_codes) return quantize_mxfp4_kernel<BF16, false, true>;
  return a.col_codes ? quantize_mxfp4_kernel<BF16, true, true> : quantize_mxfp4_kernel<BF16, true, false>;
}

}  // namespace
}  // namespace forge

using namespace forge;

extern "C" {

FORGE_API forge_status forge_quantize_mxfp4(const void* x, forge_dtype x_dtype, int64_t R,
                                            int64_t C, void* row_codes, void* row_scales,
                                            void* col_codes, void* col_scales, void* stream) {
  if (forge_status s = validate_quantize_mxfp4(x, x_dtype, R, C, row_codes, row_scales, col_codes,
                                               col_scales))
    return s;
  if (R == 0 || C == 0) return FORGE_OK;
  if (forge_status s = check_device()) return s;
  (void)hipGetLastError();
  QuantArgs a{};
  a.x = x;
  a.row_codes = static_cast<uint8_t*>(row_codes);
  a.row_scales = static_cast<uint8_t*>(row_scales);
  a.col_codes = static_cast<uint8_t*>(col_codes);
  a.col_scales = static_cast<uint8_t*>(col_scales);
  a.R = R;
  a.C = C;
  a.padded_c = FORGE_MXFP4_K(C);
  // Padding columns of the codes along rows belong to tiles too.
  const int64_t tc = x_dtype == FORGE_BF16 ? kQuantCols<true> : kQuantCols<false>;
  const int64_t across = ((row_codes ? FORGE_MXFP4_K(C) : C) + tc - 1) / tc;
  const int64_t tiles = (R + kQuantRows - 1) / kQuantRows * across;
  if (tiles >= int64_t(1) << 31) return FORGE_ERR_SHAPE;
  a.tiles_c = uint32_t(across);
  a.tiles = uint32_t(tiles);
  const dim3 grid(std::min(a.tiles, kQuantGrid));
  const auto kernel = x_dtype == FORGE_BF16 ? quantize_kernel<true>(a) : quantize_kernel<false>(a);
  hipLaunchKernelGGL(kernel, grid, dim3(kQuantThreads), 0, static_cast<hipStream_t>(stream), a);
  return launch_status();
}

FORGE_API forge_status forge_matmul_mxfp4(const void* a_codes, const void* a_scales,
                                          const void* b_codes, const void* b_scales, void* out,
                                          forge_dtype out_dtype, int64_t M, int64_t N, int64_t Kp,
                                          forge_tile tile, void* stream) {
  if (forge_status s = validate_matmul_mxfp4(a_codes, a_scales, b_codes, b_scales, out, out_dtype,
                                             M, N, Kp, tile))
    return s;
  if (M == 0 || N == 0) return FORGE_OK;
  if (forge_status s = check_device()) return s;
  if (!grid_fits(N, M, FORGE_TILE_128x128, 1)) return FORGE_ERR_SHAPE;
  if (tile == FORGE_TILE_DEFAULT) tile = choose_tile(N, M, Kp);
  (void)hipGetLastError();
  const WgradArgs a = base_args(b_codes, a_codes, static_cast<float*>(out), nullptr, nullptr, Kp, N, M);
  const MxArgs x{static_cast<const uint8_t*>(b_scales), static_cast<const uint8_t*>(a_scales), Kp};
  const hipStream_t st = static_cast<hipStream_t>(stream);
  return out_dtype == FORGE_BF16 ? MxLaunch<EPI_GRAD | EPI_BF16_OUT>::run(a, x, tile, st)
                                 : MxLaunch<EPI_GRAD>::run(a, x, tile, st);
}

FORGE_API forge_status forge_wgrad_adamw_mxfp4(const void* x_codes, const void* x_scales,
                                               const void* dy_codes, const void* dy_scales,
                                               float* W, float* m, float* v, int64_t Kp,
                                               int64_t d_in, int64_t d_out,
                                               const forge_adamw_params* p, forge_tile tile,
                                               void* stream) {
  if (forge_status s = validate_wgrad_adamw_mxfp4(x_codes, x_scales, dy_codes, dy_scales, W, m, v,
                                                  Kp, d_in, d_out, p, tile))
    return s;
  if (d_in == 0 || d_out == 0) return FORGE_OK;
  if (forge_status s = check_device()) return s;
  if (!grid_fits(d_in, d_out, FORGE_TILE_128x128, 1)) return FORGE_ERR_SHAPE;
  if (tile == FORGE_TILE_DEFAULT) tile = choose_tile(d_in, d_out, Kp);
  (void)hipGetLastError();
  WgradArgs a = base_args(x_codes, dy_codes, W, m, v, Kp, d_in, d_out);
  a.adam = make_adamw(*p);
  const MxArgs x{static_cast<const uint8_t*>(x_scales), static_cast<const uint8_t*>(dy_scales), Kp};
  return with_adamw_epi<MxLaunch>(*p, a, x, tile, static_cast<hipStream_t>(stream));
}

}  // extern "C"
