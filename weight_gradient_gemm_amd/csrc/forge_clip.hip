// Global gradient norm, clipped gradients and clipped optimizer steps over a
// list of tensors: validation, packing of the lists into launches.
#include <algorithm>
#include <climits>
#include <cstring>
#include <type_traits>

#include "clip_kernels.hpp"
#include "forge_ops.h"
#include "host.hpp"
#include "validate_ops.hpp"

namespace forge {
namespace {

// Cuts the list into tables of at most Table::N tensors and MAX_CHUNKS chunks
// and hands each to `launch(table)`; a tensor of more chunks goes into several.
template <class Table, int64_t MAX_CHUNKS, class Fill, class Launch>
forge_status for_tables(const forge_tensor* tensors, int32_t count, const Fill& fill,
                        const Launch& launch) {
  Table tab;
  int used = 0;
  int64_t chunks = 0;
  auto flush = [&]() -> forge_status {
    if (used == 0) return FORGE_OK;
    for (int t = used; t <= Table::N; ++t) tab.first[t] = INT_MAX;
    tab.chunks = int32_t(chunks);
    const forge_status s = launch(tab);
    used = 0;
    chunks = 0;
    return s;
  };
  std::memset(&tab, 0, sizeof(tab));
  for (int32_t i = 0; i < count; ++i) {
    for (int64_t at = 0; at < tensors[i].n;) {
      if (used == Table::N || chunks == MAX_CHUNKS)
        if (forge_status s = flush()) return s;
      const int64_t n = std::min(tensors[i].n - at, (MAX_CHUNKS - chunks) * kChunk);
      fill(tab, used, tensors[i], at);
      tab.tail.set(used, uint32_t((n - 1) % kChunk + 1) | (tensors[i].grad_dtype == FORGE_BF16 ? 0x8000u : 0u));
      tab.first[used] = int32_t(chunks);
      ++used;
      chunks += (n + kChunk - 1) / kChunk;
      at += n;
    }
  }
  return flush();
}

template <int OP>
forge_status launch_steps(const forge_tensor* tensors, int32_t count, const float* coef,
                          const AdamWConsts& ac, const SgdmConsts& sc, hipStream_t s) {
  constexpr bool ADAM = OP == CLIP_ADAMW || OP == CLIP_ADAMW_EXACT;
  typedef typename std::conditional<ADAM, AdamTable, ClipTable>::type Table;
  // One workgroup of 256 per chunk: the launch's work items stay below 2^32.
  return for_tables<Table, (int64_t(1) << 23)>(
      tensors, count,
      [](Table& tab, int k, const forge_tensor& t, int64_t at) {
        const int64_t gb = at * dtype_bytes(t.grad_dtype);
        tab.set(0, k, t.grad, gb);
        if constexpr (OP == CLIP_SCALE) tab.set(1, k, t.out, gb);
        if constexpr (OP != CLIP_SCALE) {
          tab.set(1, k, t.W, at * 4);
          tab.set(2, k, t.m, at * 4);
        }
        if constexpr (ADAM) tab.set(3, k, t.v, at * 4);
      },
      [&](const Table& tab) {
        hipLaunchKernelGGL((clip_step_kernel<OP, Table>), dim3(tab.chunks), dim3(256), 0, s, tab,
                           coef, ac, sc);
        return launch_status();
      });
}

bool all_empty(const forge_tensor* tensors, int32_t count) {
  for (int32_t i = 0; i < count; ++i)
    if (tensors[i].n > 0) return false;
  return true;
}

}  // namespace
}  // namespace forge

using namespace forge;

extern "C" {

FORGE_API int64_t forge_grad_norm_workspace(int32_t count) { return grad_norm_workspace(count); }

FORGE_API forge_status forge_grad_norm(const forge_tensor* tensors, int32_t count,
                                       double max_norm, float* norm_coef, void* workspace,
                                       int64_t workspace_bytes, void* stream) {
  if (forge_status s = validate_grad_norm(tensors, count, max_norm, norm_coef, workspace,
                                          workspace_bytes))
    return s;
  if (forge_status s = check_device()) return s;
  (void)hipGetLastError();
  const hipStream_t st = static_cast<hipStream_t>(stream);
  double* const part = static_cast<double*>(workspace);
  int64_t parts = 0;
  bool alone = false;
  const forge_status s = for_tables<NormTable, kMaxListElems / kChunk + FORGE_MAX_TENSORS>(
      tensors, count,
      [](NormTable& tab, int k, const forge_tensor& t, int64_t at) {
        tab.set(0, k, t.grad, at * dtype_bytes(t.grad_dtype));
      },
      [&](const NormTable& tab) {
        // A short list of few tensors: one workgroup, one launch.
        alone = count <= kNormTensors && tab.chunks <= kNormAlone;
        if (alone) {
          hipLaunchKernelGGL(norm_alone_kernel, dim3(1), dim3(1024), 0, st, tab, max_norm,
                             norm_coef);
          return launch_status();
        }
        const int grid = std::min(int(tab.chunks), kNormGrid);
        hipLaunchKernelGGL(norm_partial_kernel, dim3(grid), dim3(256), 0, st, tab, part + parts);
        parts += grid;
        return launch_status();
      });
  if (s || alone) return s;
  hipLaunchKernelGGL(norm_finish_kernel, dim3(1), dim3(1024), 0, st, part, parts, max_norm,
                     norm_coef);
  return launch_status();
}

FORGE_API forge_status forge_clip_grads(const forge_tensor* tensors, int32_t count,
                                        const float* coef, void* stream) {
  if (forge_status s = validate_clip_grads(tensors, count, coef)) return s;
  if (all_empty(tensors, count)) return FORGE_OK;
  if (forge_status s = check_device()) return s;
  (void)hipGetLastError();
  return launch_steps<CLIP_SCALE>(tensors, count, coef, AdamWConsts{}, SgdmConsts{},
                                  static_cast<hipStream_t>(stream));
}

FORGE_API forge_status forge_adamw_clipped(const forge_tensor* tensors, int32_t count,
                                           const float* coef, const forge_adamw_params* p,
                                           void* stream) {
  if (forge_status s = validate_adamw_clipped(tensors, count, coef, p)) return s;
  if (all_empty(tensors, count)) return FORGE_OK;
  if (forge_status s = check_device()) return s;
  (void)hipGetLastError();
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const AdamWConsts ac = make_adamw(*p);
  return p->eps > 0.0 ? launch_steps<CLIP_ADAMW>(tensors, count, coef, ac, SgdmConsts{}, st)
                      : launch_steps<CLIP_ADAMW_EXACT>(tensors, count, coef, ac, SgdmConsts{}, st);
}

FORGE_API forge_status forge_sgdm_clipped(const forge_tensor* tensors, int32_t count,
                                          const float* coef, const forge_sgdm_params* p,
                                          void* stream) {
  if (forge_status s = validate_sgdm_clipped(tensors, count, coef, p)) return s;
  if (all_empty(tensors, count)) return FORGE_OK;
  if (forge_status s = check_device()) return s;
  (void)hipGetLastError();
  return launch_steps<CLIP_SGDM>(tensors, count, coef, AdamWConsts{}, make_sgdm(*p),
                                 static_cast<hipStream_t>(stream));
}

}  // extern "C"
