// Layer norm entry points of the forge C ABI.
#include <algorithm>
#include <cstdint>

#include "forge_ops.h"
#include "host.hpp"
#include "layernorm_kernels.hpp"
#include "validate_ops.hpp"

namespace forge {
namespace {

static_assert(kLayernormParts <= 8 * kLnReduceGroups, "parts that the last sum reads");

// Most workgroups of a launch over rows that registers do not hold; what is beyond loops.
// A few to a CU that loop take longer: 20000 x 16392 bf16 forward 345 us, with 1, 2 and 4 to
// a CU 440, 391 and 382, 8192 x 24576 197 and 255, 226, 222; backward 3 to 5% longer.
constexpr int64_t kMaxGrid = int64_t(1) << 20;

dim3 grid_for(int64_t blocks) { return dim3(uint32_t(std::min(blocks, kMaxGrid))); }

template <bool XB, bool YB, int EL, int WAVES>
forge_status launch_forward(const LnArgs& a, hipStream_t s) {
  const int64_t blocks = (a.T + ln_rows<WAVES> - 1) / ln_rows<WAVES>;
  const int64_t most = int64_t(std::max(16, persistent_grid())) * (WAVES == 8 ? 2 : 6);
  hipLaunchKernelGGL((layernorm_kernel<XB, YB, EL, WAVES>), dim3(uint32_t(std::min(blocks, most))),
                     dim3(ln_threads<WAVES>), 0, s, a);
  return launch_status();
}

template <bool XB, bool YB>
struct Forward {
  static forge_status run(const LnArgs& a, hipStream_t s) {
    if (a.d <= 512) return launch_forward<XB, YB, 8, 1>(a, s);
    if (a.d <= 1024) return launch_forward<XB, YB, 16, 1>(a, s);
    if (a.d <= 2048) return launch_forward<XB, YB, 8, 4>(a, s);
    if (a.d <= 4096) return launch_forward<XB, YB, 16, 4>(a, s);
    if (a.d <= 8192) return launch_forward<XB, YB, 32, 4>(a, s);
    if (a.d <= 16384) return launch_forward<XB, YB, 32, 8>(a, s);
    hipLaunchKernelGGL((layernorm_wide_kernel<XB, YB>), grid_for(a.T), dim3(1024), 0, s, a);
    return launch_status();
  }
};

// Workgroups: what is added up behind them grows with their number. One to a CU of
// more than four waves (4096 x 16384 bf16 92 us, with two 104). Of four waves two to a CU
// where there is work for many rounds: 4000 x 4096 bf16 31 us, with one 33, float32 44.7 and 45.6;
// 2800 rows 27.1 and 26.7, 36.4 and 35.4; 3500 x 5000 bf16 37 and 41. Rows of more than 4096
// columns gain later or not at all where they are float32: x alone, 4096 x 8192 69 and
// 65, 8192 x 5000 88 and 90; both, 8192 x 5000 100 and 94, 8192 x 8192 144 and 138. Half as
// many as CUs for few rows (256 x 4096 8.9 and 10.8).
template <bool XB, bool YB, int EL, int WAVES, int ROWS>
forge_status launch_backward(const LnArgs& a, int32_t& parts, hipStream_t s) {
  const int64_t rounds = (a.T + ROWS - 1) / ROWS;
  const int64_t many = EL <= 16 || (XB && YB) ? 3500 : XB || YB ? 4096 : INT64_MAX;
  const int64_t most = WAVES * ROWS > 4 ? kLayernormParts / 2
                       : rounds >= many ? kLayernormParts
                       : rounds >= 512  ? kLayernormParts / 2
                                        : kLayernormParts / 4;
  parts = int32_t(std::min(rounds, most));
  hipLaunchKernelGGL((layernorm_backward_kernel<XB, YB, EL, WAVES, ROWS>), dim3(parts),
                     dim3(64 * WAVES * ROWS), 0, s, a);
  return launch_status();
}

template <bool XB, bool YB>
struct Backward {
  static forge_status run(const LnArgs& a, int32_t& parts, hipStream_t s) {
    if (a.d <= 512) return launch_backward<XB, YB, 8, 1, 4>(a, parts, s);
    if (a.d <= 1024) return launch_backward<XB, YB, 16, 1, 4>(a, parts, s);
    if (a.d <= 2048) return launch_backward<XB, YB, 8, 4, 4>(a, parts, s);
    if (a.d <= 4096) return launch_backward<XB, YB, 16, 4, 1>(a, parts, s);
    if (a.d <= 8192) return launch_backward<XB, YB, 32, 4, 1>(a, parts, s);
    if (a.d <= 16384) return launch_backward<XB, YB, 32, 8, 1>(a, parts, s);
    // Sums of so many columns do not fit a workgroup's registers beside the row:
    // the columns first, as dX may overwrite dY.
    constexpr int E = io_elems<XB, YB>;
    parts = int32_t(std::min<int64_t>((a.T + 8 * kLnColumnRows - 1) / (8 * kLnColumnRows), 64));
    hipLaunchKernelGGL((layernorm_columns_kernel<XB, YB>), dim3((a.d + 32 * E - 1) / (32 * E), parts),
                       dim3(256), 0, s, a);
    if (forge_status st = launch_status()) return st;
    hipLaunchKernelGGL((layernorm_dx_wide_kernel<XB, YB>), grid_for(a.T), dim3(1024), 0, s, a);
    return launch_status();
  }
};

// F of the element types of x and y.
template <template <bool, bool> class F, class... Args>
forge_status with_types(forge_dtype x, forge_dtype y, Args&&... args) {
  if (x == FORGE_BF16)
    return y == FORGE_BF16 ? F<true, true>::run(args...) : F<true, false>::run(args...);
  return y == FORGE_BF16 ? F<false, true>::run(args...) : F<false, false>::run(args...);
}

}  // namespace
}  // namespace forge

using namespace forge;

extern "C" {

FORGE_API forge_status forge_layernorm(const void* x, forge_dtype x_dtype, const float* gamma,
                                       const float* beta, void* y, forge_dtype y_dtype, float* mean,
                                       float* rstd, int64_t T, int64_t d, double eps, void* stream) {
  if (forge_status s = validate_layernorm(x, x_dtype, gamma, beta, y, y_dtype, mean, rstd, T, d, eps))
    return s;
  if (T == 0 || d == 0) return FORGE_OK;
  if (forge_status s = check_device()) return s;
  (void)hipGetLastError();
  LnArgs a{};
  a.x = x;
  a.gamma = gamma;
  a.beta = beta;
  a.out = y;
  a.mean = mean;
  a.rstd = rstd;
  a.T = T;
  a.d = int32_t(d);
  a.eps = float(eps);
  return with_types<Forward>(x_dtype, y_dtype, a, static_cast<hipStream_t>(stream));
}

FORGE_API int64_t forge_layernorm_workspace(int64_t T, int64_t d) { return layernorm_workspace(T, d); }

FORGE_API forge_status forge_layernorm_backward(const void* dY, forge_dtype y_dtype, const void* x,
                                                forge_dtype x_dtype, const float* gamma,
                                                const float* mean, const float* rstd, void* dX,
                                                float* dgamma, float* dbeta, int64_t T, int64_t d,
                                                void* workspace, int64_t workspace_bytes,
                                                void* stream) {
  if (forge_status s = validate_layernorm_backward(dY, y_dtype, x, x_dtype, gamma, mean, rstd, dX,
                                                   dgamma, dbeta, T, d, workspace, workspace_bytes))
    return s;
  if (d == 0) return FORGE_OK;
  if (forge_status s = check_device()) return s;
  (void)hipGetLastError();
  const hipStream_t st = static_cast<hipStream_t>(stream);
  int32_t parts = 0;
  if (T > 0) {
    LnArgs a{};
    a.x = x;
    a.dy = dY;
    a.gamma = gamma;
    a.out = dX;
    a.mean = const_cast<float*>(mean);
    a.rstd = const_cast<float*>(rstd);
    a.part = static_cast<float*>(workspace);
    a.T = T;
    a.d = int32_t(d);
    if (forge_status s = with_types<Backward>(x_dtype, y_dtype, a, parts, st)) return s;
  }
  const LnReduce r{static_cast<const float*>(workspace), dgamma, dbeta, int32_t(d), parts,
                   int32_t(dbeta ? 2 * d : d)};
  hipLaunchKernelGGL(layernorm_reduce_kernel, dim3((r.columns + kLnReduceColumns - 1) / kLnReduceColumns),
                     dim3(8 * kLnReduceGroups), 0, st, r);
  return launch_status();
}

}  // extern "C"
