// Embedding lookup and gradient entry points of the forge C ABI.
#include <algorithm>

#include "embedding_kernels.hpp"
#include "forge_ops.h"
#include "host.hpp"
#include "validate_ops.hpp"

namespace forge {
namespace {

// Most workgroups of 256 threads of a launch; what is beyond loops.
constexpr int64_t kMaxGrid = int64_t(1) << 22;
constexpr int64_t kMaxBlocks = int64_t(1) << 31;
// Lookups of so many bytes do not leave their output in the caches.
constexpr int64_t kStreamBytes = int64_t(1) << 27;

// `count` rows of `units` each, and their workgroups of 256 * pieces units.
// False if they do not fit 31 bits (far more than memory holds).
template <class Args>
bool cut_rows(Args& a, int64_t count, int64_t units, int64_t pieces = 1) {
  a.rows.units = uint32_t(units);
  a.rows.magic = uint32_t(((int64_t(1) << 20) + units - 1) / units);
  const int64_t blocks = (count * units + 256 * pieces - 1) / (256 * pieces);
  a.blocks = uint32_t(blocks);
  return blocks < kMaxBlocks;
}

dim3 grid_for(int64_t blocks) { return dim3(uint32_t(std::min(blocks, kMaxGrid))); }

int bits_for(int64_t largest) {
  int b = 1;
  while ((int64_t(1) << b) <= largest) ++b;
  return b;
}

template <bool DIRECT>
forge_status launch_sort_pass(const SortPass& p, hipStream_t s) {
  const dim3 grid(p.tiles), threads(kTileThreads);
  hipLaunchKernelGGL((sort_count_kernel<DIRECT>), grid, threads, 0, s, p);
  if (forge_status st = launch_status()) return st;
  if (!DIRECT) {
    hipLaunchKernelGGL(sort_sum_kernel, dim3(1u << p.bits), threads, 0, s, p);
    if (forge_status st = launch_status()) return st;
  }
  hipLaunchKernelGGL((sort_scatter_kernel<DIRECT>), grid, threads, 0, s, p);
  return launch_status();
}

// Sorts the tokens by row into a.keys, a.pos.
forge_status launch_sort(const IdSource& src, const EmbeddingWorkspace& ws, char* base, int64_t T,
                         EmbeddingArgs& a, hipStream_t s) {
  uint32_t* const keys[2] = {reinterpret_cast<uint32_t*>(base + ws.keys[0]),
                             reinterpret_cast<uint32_t*>(base + ws.keys[1])};
  uint32_t* const pos[2] = {reinterpret_cast<uint32_t*>(base + ws.pos[0]),
                            reinterpret_cast<uint32_t*>(base + ws.pos[1])};
  a.keys = keys[0];
  a.pos = pos[0];
  const int key_bits = bits_for(src.V);
  if (T <= kRankTokens) {
    hipLaunchKernelGGL(rank_kernel, dim3(uint32_t(T + kRankKeys - 1) / kRankKeys), dim3(8 * kRankKeys),
                       0, s, src, int(T), keys[0], pos[0]);
    return launch_status();
  }
  const int passes = (key_bits + kDigitBits - 1) / kDigitBits;
  SortPass p{};
  p.src = src;
  p.count = reinterpret_cast<uint32_t*>(base + ws.count);
  p.T = T;
  p.tiles = int32_t((T + kTileKeys - 1) / kTileKeys);
  p.total = p.count + int64_t(p.tiles) * kDigits;
  for (int k = 0; k < passes; ++k) {
    p.keys_in = k ? keys[(k - 1) & 1] : nullptr;
    p.pos_in = k ? pos[(k - 1) & 1] : nullptr;
    p.keys_out = keys[k & 1];
    p.pos_out = pos[k & 1];
    p.shift = key_bits * k / passes;
    p.bits = key_bits * (k + 1) / passes - p.shift;
    const forge_status st =
        p.tiles <= kDirectTiles ? launch_sort_pass<true>(p, s) : launch_sort_pass<false>(p, s);
    if (st) return st;
  }
  a.keys = p.keys_out;
  a.pos = p.pos_out;
  return FORGE_OK;
}

template <int OP, bool BF16>
forge_status launch_gradient_t(EmbeddingArgs a, hipStream_t s) {
  EmbeddingArgs b = a;
  b.bound_blocks = uint32_t(a.V + 256) / 256;
  b.slices = uint32_t(a.d / 4 + 255) / 256;
  b.blocks = b.bound_blocks + uint32_t(a.T >> a.chunk_bits) * b.slices;
  hipLaunchKernelGGL((embedding_bounds_kernel<BF16>), grid_for(b.blocks), dim3(256), 0, s, b);
  if (forge_status st = launch_status()) return st;
  hipLaunchKernelGGL((embedding_rows_kernel<OP, BF16>), grid_for(a.blocks), dim3(256), 0, s, a);
  return launch_status();
}

// Few tokens: up to four pieces to a workgroup, so that looking through the ids
// is small beside its rows' traffic, but not so many that the chip stands idle.
template <int OP, bool BF16>
forge_status launch_scan(EmbeddingArgs a, const IdSource& src, hipStream_t s) {
  a.scan_units = uint32_t(std::max<int64_t>(1, std::min<int64_t>(kScanUnits, a.blocks / 1024)));
  (void)cut_rows(a, a.V, a.d / 4, a.scan_units);
  hipLaunchKernelGGL((embedding_scan_kernel<OP, BF16>), grid_for(a.blocks), dim3(kScanTokens), 0, s,
                     a, src);
  return launch_status();
}

template <int OP>
forge_status launch_gradient(const void* ids, int32_t id_bytes, const void* dY, forge_dtype dY_dtype,
                             EmbeddingArgs a, void* workspace, void* stream) {
  if (forge_status s = check_device()) return s;
  (void)hipGetLastError();
  if (!cut_rows(a, a.V, a.d / 4) || (a.T >> a.chunk_bits) * (a.d / 1024 + 1) >= kMaxBlocks)
    return FORGE_ERR_SHAPE;
  const hipStream_t st = static_cast<hipStream_t>(stream);
  const IdSource src{ids, id_bytes, uint32_t(a.V)};
  a.dY = dY;
  const bool bf16 = dY_dtype == FORGE_BF16;
  if (a.T <= kScanTokens)
    return bf16 ? launch_scan<OP, true>(a, src, st) : launch_scan<OP, false>(a, src, st);
  const EmbeddingWorkspace ws = embedding_workspace(a.T, a.V, a.d);
  char* const base = static_cast<char*>(workspace);
  a.bound = reinterpret_cast<uint32_t*>(base + ws.bound);
  a.chunk = reinterpret_cast<float*>(base + ws.chunk);
  if (forge_status s = launch_sort(src, ws, base, a.T, a, st)) return s;
  return bf16 ? launch_gradient_t<OP, true>(a, st) : launch_gradient_t<OP, false>(a, st);
}

template <bool STREAM>
void (*lookup_kernel(forge_dtype table, forge_dtype out))(LookupArgs) {
  if (table == FORGE_BF16)
    return out == FORGE_BF16 ? embedding_kernel<true, true, STREAM> : embedding_kernel<true, false, STREAM>;
  return out == FORGE_BF16 ? embedding_kernel<false, true, STREAM> : embedding_kernel<false, false, STREAM>;
}

EmbeddingArgs gradient_args(float* W, float* m, float* v, int64_t T, int64_t V, int64_t d,
                            double scale) {
  EmbeddingArgs a{};
  a.W = W;
  a.m = m;
  a.v = v;
  a.T = T;
  a.V = int32_t(V);
  a.d = int32_t(d);
  a.chunk_bits = embedding_chunk_bits(T);
  a.scale = float(scale);
  return a;
}

}  // namespace
}  // namespace forge

using namespace forge;

extern "C" {

FORGE_API forge_status forge_embedding(const void* table, forge_dtype table_dtype,
                                       const void* ids, int32_t id_bytes, void* out,
                                       forge_dtype out_dtype, int64_t T, int64_t V, int64_t d,
                                       double scale, void* stream) {
  if (forge_status s = validate_embedding(table, table_dtype, ids, id_bytes, out, out_dtype, T, V,
                                          d, scale))
    return s;
  if (T == 0 || d == 0) return FORGE_OK;
  if (forge_status s = check_device()) return s;
  (void)hipGetLastError();
  LookupArgs a{};
  a.src = IdSource{ids, id_bytes, uint32_t(V)};
  a.table = table;
  a.out = out;
  a.T = T;
  a.d = int32_t(d);
  a.scale = float(scale);
  if (!cut_rows(a, T, d / 8)) return FORGE_ERR_SHAPE;
  const bool stream_out = T * d * dtype_bytes(out_dtype) >= kStreamBytes;
  const auto kernel = stream_out ? lookup_kernel<true>(table_dtype, out_dtype)
                                 : lookup_kernel<false>(table_dtype, out_dtype);
  hipLaunchKernelGGL(kernel, grid_for(a.blocks), dim3(256), 0, static_cast<hipStream_t>(stream), a);
  return launch_status();
}

FORGE_API int64_t forge_embedding_workspace(int64_t T, int64_t V, int64_t d) {
  return embedding_sizes_ok(T, V, d) ? embedding_workspace(T, V, d).bytes : 0;
}

FORGE_API forge_status forge_embedding_grad(const void* ids, int32_t id_bytes, const void* dY,
                                            forge_dtype dY_dtype, float* grad, int64_t T,
                                            int64_t V, int64_t d, double scale,
                                            int32_t accumulate, void* workspace,
                                            int64_t workspace_bytes, void* stream) {
  const void* outs[1] = {grad};
  if (forge_status s = validate_embedding_grad(ids, id_bytes, dY, dY_dtype, outs, 1, T, V, d,
                                               scale, workspace, workspace_bytes))
    return s;
  if (V == 0 || d == 0) return FORGE_OK;
  const EmbeddingArgs a = gradient_args(grad, nullptr, nullptr, T, V, d, scale);
  return accumulate
             ? launch_gradient<EMB_GRAD_ADD>(ids, id_bytes, dY, dY_dtype, a, workspace, stream)
             : launch_gradient<EMB_GRAD>(ids, id_bytes, dY, dY_dtype, a, workspace, stream);
}

FORGE_API forge_status forge_embedding_adamw(const void* ids, int32_t id_bytes, const void* dY,
                                             forge_dtype dY_dtype, float* W, float* m, float* v,
                                             int64_t T, int64_t V, int64_t d, double scale,
                                             const forge_adamw_params* p, void* workspace,
                                             int64_t workspace_bytes, void* stream) {
  const void* outs[3] = {W, m, v};
  if (!p) return FORGE_ERR_NULL;
  if (forge_status s = validate_embedding_grad(ids, id_bytes, dY, dY_dtype, outs, 3, T, V, d,
                                               scale, workspace, workspace_bytes))
    return s;
  if (forge_status s = check_adamw_params(p)) return s;
  if (V == 0 || d == 0) return FORGE_OK;
  EmbeddingArgs a = gradient_args(W, m, v, T, V, d, scale);
  a.adam = make_adamw(*p);
  return p->eps > 0.0
             ? launch_gradient<EMB_ADAMW>(ids, id_bytes, dY, dY_dtype, a, workspace, stream)
             : launch_gradient<EMB_ADAMW_EXACT>(ids, id_bytes, dY, dY_dtype, a, workspace, stream);
}

FORGE_API forge_status forge_embedding_sgdm(const void* ids, int32_t id_bytes, const void* dY,
                                            forge_dtype dY_dtype, float* W, float* mom, int64_t T,
                                            int64_t V, int64_t d, double scale,
                                            const forge_sgdm_params* p, void* workspace,
                                            int64_t workspace_bytes, void* stream) {
  const void* outs[2] = {W, mom};
  if (!p) return FORGE_ERR_NULL;
  if (forge_status s = validate_embedding_grad(ids, id_bytes, dY, dY_dtype, outs, 2, T, V, d,
                                               scale, workspace, workspace_bytes))
    return s;
  if (forge_status s = check_sgdm_params(p)) return s;
  if (V == 0 || d == 0) return FORGE_OK;
  EmbeddingArgs a = gradient_args(W, mom, nullptr, T, V, d, scale);
  a.sgd = make_sgdm(*p);
  return launch_gradient<EMB_SGDM>(ids, id_bytes, dY, dY_dtype, a, workspace, stream);
}

}  // extern "C"
