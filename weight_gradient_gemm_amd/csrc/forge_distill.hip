// Distillation entry points of the forge C ABI.
#include <algorithm>

#include "distill_kernels.hpp"
#include "forge_ops.h"
#include "host.hpp"
#include "validate_ops.hpp"

namespace forge {
namespace {

static_assert(kDistillMaxK == FORGE_DISTILL_MAX_K && kDistillChunk == kChunkColumns &&
                  kDistillHeld == 1024 * 16 * kVec<true> && kDistillHeld == 2 * 1024 * 16 * kVec<false>,
              "the kernels' sizes");

// A chunk to a workgroup: 2^20 at most, of rows of up to 2^22 columns.
static_assert(kDistillChunkRows * ((int64_t(1) << 22) / kDistillChunk) <= int64_t(1) << 20, "workgroups of a launch");

template <bool ZB, bool GB, int THREADS, int NV>
forge_status launch_rows_t(const DistillArgs& a, int per_cu, hipStream_t s) {
  const int64_t grid = int64_t(std::max(16, persistent_grid())) * per_cu;
  hipLaunchKernelGGL((distill_rows_kernel<ZB, GB, THREADS, NV>), dim3(uint32_t(std::min(grid, a.T))),
                     dim3(THREADS), 0, s, a);
  return launch_status();
}

template <bool ZB, bool GB>
forge_status launch_rows(const DistillArgs& a, hipStream_t s) {
  constexpr int E = kVec<ZB>;
  if (a.V <= 256 * 4 * E) return launch_rows_t<ZB, GB, 256, 4>(a, 5, s);
  if (a.V <= 512 * 8 * E) return launch_rows_t<ZB, GB, 512, 8>(a, 2, s);
  if (a.V <= 512 * 16 * E) return launch_rows_t<ZB, GB, 512, 16>(a, 2, s);
  return launch_rows_t<ZB, GB, 1024, 16>(a, 1, s);
}

template <bool ZB, bool GB>
forge_status launch_chunks(DistillArgs a, hipStream_t s) {
  a.items = a.T * a.chunks;
  if (a.items > 0 && a.K > 0) {
    hipLaunchKernelGGL((distill_stats_kernel<ZB>), dim3(uint32_t(a.items)), dim3(kChunkThreads), 0, s, a);
    if (forge_status st = launch_status()) return st;
  }
  a.items = a.T * a.chunks_out;
  hipLaunchKernelGGL((distill_gradient_kernel<ZB, GB>), dim3(uint32_t(a.items)), dim3(kChunkThreads), 0, s, a);
  return launch_status();
}

// A row to a workgroup, or chunks of it (distill_in_chunks). Chunks take a launch
// more (3 us) and read the logits twice, but a workgroup takes 5 us and one more for each 7000
// columns with a row (for each 3500 where it does not hold it), however few there are: bf16
// 8 x 128256 7.6 us in chunks and 21 by rows, 64 x 128256 16 and 22, 96 x 128256 22 and 23, 128 x
// 128256 26 and 23, 96 x 32000 10.5 and 10.6, 8 x 8192 7.8 and 6.6. The loss alone: 8 x 128256
// 6.3 us in chunks and 10.0 by rows, 96 x 128256 11.0 and 10.9, 8 x 60000 6.5 and 6.5.
//
// Rows that are not held run one to a CU, and a last round of 256 of them takes half of a round
// however few they are, where chunks take time by the row. So the rows of the last round
// count: float32 with a bf16 gradient, 128256 columns, 128 rows 33 us in chunks and 45 by
// rows, 256 55 and 55; 257 56 and 82, 448 95 and 104, 512 108 and 110; 513 108 and 134, 640 144 and
// 150, 700 158 and 156 (100000 columns: 224 rows 40 and 39, 512 86 and 82, 700 118 and 116).
// Where most of the row is held (70000 columns: 128 rows 22 and 23, 192 29 and 26, 352 45 and 46,
// 384 48 and 47, 560 67 and 69, 600 72 and 71) and for bf16 (200000: 128 37 and 44, 192 49 and 48,
// 384 89 and 90, 400 93 and 91, 513 120 and 131, 600 136 and 136) rows catch up earlier.
template <bool ZB, bool GB>
forge_status launch(const DistillArgs& a, hipStream_t s) {
  if (distill_in_chunks(a.T, a.V, ZB, a.grad != nullptr)) return launch_chunks<ZB, GB>(a, s);
  if (a.grad) return launch_rows<ZB, GB>(a, s);
  const int64_t grid = int64_t(std::max(16, persistent_grid())) * 3;
  hipLaunchKernelGGL((distill_loss_kernel<ZB>), dim3(uint32_t(std::min(grid, a.T))), dim3(kLossThreads), 0, s, a);
  return launch_status();
}

}  // namespace
}  // namespace forge

using namespace forge;

extern "C" {

FORGE_API int64_t forge_distill_workspace(int64_t T, int64_t V, int64_t K) {
  return distill_sizes_ok(T, V, K) ? distill_workspace(T, V, K).bytes : 0;
}

FORGE_API forge_status forge_distill(const void* logits, forge_dtype z_dtype, int64_t ld,
                                     const void* teacher, forge_dtype teacher_dtype, const void* ids,
                                     int32_t id_bytes, const float* weight, float* loss, void* grad,
                                     forge_dtype grad_dtype, int64_t T, int64_t V, int64_t K,
                                     double temperature, double scale, void* workspace,
                                     int64_t workspace_bytes, void* stream) {
  if (forge_status s = validate_distill(logits, z_dtype, ld, teacher, teacher_dtype, ids, id_bytes,
                                        weight, loss, grad, grad_dtype, T, V, K, temperature, scale,
                                        workspace, workspace_bytes))
    return s;
  if (T == 0) return FORGE_OK;
  if (forge_status s = check_device()) return s;
  (void)hipGetLastError();
  const DistillWorkspace ws = distill_workspace(T, V, K);
  char* const base = static_cast<char*>(workspace);
  DistillArgs a{};
  a.z = logits;
  a.teacher = teacher;
  a.ids = ids;
  a.weight = weight;
  a.loss = loss;
  a.grad = grad;
  a.stats = reinterpret_cast<float2*>(base + ws.stats);
  a.logit = reinterpret_cast<float*>(base + ws.logit);
  a.T = T;
  a.ld = ld;
  a.V = int32_t(V);
  a.K = int32_t(K);
  a.chunks = int32_t((V + kDistillChunk - 1) / kDistillChunk);
  a.chunks_out = grad ? std::max(1, int32_t((ld + kDistillChunk - 1) / kDistillChunk)) : 1;
  a.wide_ids = id_bytes == 8;
  a.teacher_bf16 = teacher_dtype == FORGE_BF16;
  a.c = float(1.4426950408889634 / temperature);
  a.loss_scale = float(scale * temperature * temperature);
  a.grad_scale = float(scale * temperature);
  const hipStream_t st = static_cast<hipStream_t>(stream);
  if (z_dtype == FORGE_BF16)
    return grad_dtype == FORGE_BF16 ? launch<true, true>(a, st) : launch<true, false>(a, st);
  return grad_dtype == FORGE_BF16 ? launch<false, true>(a, st) : launch<false, false>(a, st);
}

}  // extern "C"
